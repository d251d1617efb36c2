// Rotary positions of q and k rows, in place, to other rows, or (k, with v's
// rows beside them) into the slots of a paged cache.
//
// Pages: vllm.cpp PR #26 "feat(minimax-h3)", "The device-resident forward (W2b)"
// (NeoX rotate_half) and the device-encoder commit (M-RoPE: several position
// axes); layouts, long-context scalings and slots as include/h3attn.h states them.
//
// Angles: t / 2 pi = p f / 2 pi is wanted modulo 1 only, and f / 2 pi as a fraction
// of 2^64 makes the 64-bit product p * turns[j] wrap at whole turns by itself:
// exact for every 32-bit position, no table of angles to read and no range
// reduction (p f in fp32 would be off by p 2^-24 radians, 0.06 at a million).  The
// product's top 32 bits are the angle in (-1/2, 1/2] turns for sincospi.
//
// HBM-bound: every row is read and written once.  A block takes a few tokens; it
// computes their angles once for all heads, into shared memory, and eight lanes
// take a row, two 16-byte chunks each: in the half layout the two that hold a
// rotation's pairs, so nothing is exchanged between lanes.  A lane group's first
// rows are on their way while the block computes its angles.  20,423 tokens of 32
// heads: 55 us, 6.1 TB/s, 91 % of the measured copy.
#include <algorithm>

#include "device_common.cuh"
#include "qk_norm.cuh"

namespace h3 {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 8;  // rows in work at once
constexpr int kAhead = 4;              // rows of a lane group whose loads go out together
constexpr int kMaxTokens = 16;         // of a block

__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  // (cos, sin) of pairs 8l + 2i and 8l + 2i + 1 at [token][i][l]: a row's eight lanes read 128 bytes at a time
  __shared__ float4 angle[kMaxTokens][4][8];
  __shared__ int64_t stored[kMaxTokens];  // cache offset of the token's slot, -1: none
  const int64_t tok0 = (int64_t)blockIdx.x * a.block_tokens;
  const int tokens = (int)min((int64_t)a.block_tokens, a.n - tok0);
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int half = a.rope.rope_dims / 2, pair_lanes = a.rope.rope_dims / 16;
  // this lane's chunks: half layout, a pair of chunks of the rotated dims, or two of the others; interleaved, neighbours
  int c0 = 2 * lane, c1 = c0 + 1;
  bool turns = lane < pair_lanes;
  if (!a.rope.interleaved) {
    c0 = turns ? lane : 2 * lane;
    c1 = turns ? lane + pair_lanes : c0 + 1;
  }
  const int rows = a.H + a.Hk + a.Hv, total = tokens * rows;

  struct Row {
    const __nv_bfloat16* in;
    __nv_bfloat16* out;   // null: not stored
    int tok;
    bool copy;            // v's
  };
  const auto row_of = [&](int f) {
    Row r;
    r.tok = f / rows;
    int h = f - r.tok * rows;
    const int64_t tok = tok0 + r.tok;
    r.copy = false;
    if (h < a.H) {
      r.in = a.q_in + tok * a.q_in_stride + h * kHeadDim;
      r.out = a.q_out + tok * a.q_out_stride + h * kHeadDim;
      return r;
    }
    h -= a.H;
    r.copy = h >= a.Hk;
    if (r.copy) h -= a.Hk;
    r.in = (r.copy ? a.v_in : a.k_in) + tok * a.k_in_stride + h * kHeadDim;
    r.out = (r.copy ? a.v_out : a.k_out) + (int64_t)h * a.k_out_head_stride;
    if (a.slots == nullptr) {
      r.out += tok * a.k_out_stride;
    } else if (stored[r.tok] < 0) {
      r.out = nullptr;
    } else {
      r.out += stored[r.tok];
    }
    return r;
  };
  const auto in_of = [&](int f) {  // (row_of without the slot, which is not known before the barrier)
    const int t = f / rows;
    int h = f - t * rows;
    const int64_t tok = tok0 + t;
    if (h < a.H) return a.q_in + tok * a.q_in_stride + h * kHeadDim;
    h -= a.H;
    const __nv_bfloat16* p = a.k_in;
    if (h >= a.Hk) {
      h -= a.Hk;
      p = a.v_in;
    }
    return p + tok * a.k_in_stride + h * kHeadDim;
  };

  uint4 x[kAhead], y[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int f = group + i * kGroups;
    if (f < total) {
      const uint4* p = reinterpret_cast<const uint4*>(in_of(f));
      x[i] = __ldcs(p + c0);
      y[i] = __ldcs(p + c1);
    }
  }
  for (int e = threadIdx.x; e < tokens * half; e += kThreads) {
    const int t = e / half, j = e - t * half;
    const int64_t p = __ldg(a.positions + (int64_t)a.rope.axis[j] * a.n + tok0 + t);
    const int32_t turn = (int32_t)(((uint64_t)p * a.rope.turns[j]) >> 32);
    float s, c;
    sincospif((float)turn * 4.656612873077393e-10f, &s, &c);  // 2^-31
    if (a.inverse) s = -s;
    float2* const at = reinterpret_cast<float2*>(&angle[t][(j & 7) >> 1][j >> 3]);
    at[j & 1] = make_float2(c * a.rope.amplitude, s * a.rope.amplitude);
  }
  if (a.slots != nullptr && threadIdx.x < (unsigned)tokens) {
    const int32_t slot = __ldg(a.slots + tok0 + threadIdx.x);
    int64_t at = -1;
    if (slot >= 0 && slot < a.n_slots) {
      const int32_t page = slot / a.page_size;
      at = page * a.page_stride + (int64_t)(slot - page * a.page_size) * a.k_out_stride;
    }
    stored[threadIdx.x] = at;
  }
  __syncthreads();

  for (int f0 = group; f0 < total; f0 += kAhead * kGroups) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int f = f0 + i * kGroups;
      if (f >= total) break;
      const Row r = row_of(f);
      if (turns && !r.copy) {
        float u[8], w[8];
        qkn::unpack8(x[i], u);
        qkn::unpack8(y[i], w);
        if (!a.rope.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 cs = angle[r.tok][e][lane];
            const float u0 = u[2 * e], u1 = u[2 * e + 1], w0 = w[2 * e], w1 = w[2 * e + 1];
            u[2 * e] = fmaf(u0, cs.x, -w0 * cs.y);
            w[2 * e] = fmaf(w0, cs.x, u0 * cs.y);
            u[2 * e + 1] = fmaf(u1, cs.z, -w1 * cs.w);
            w[2 * e + 1] = fmaf(w1, cs.z, u1 * cs.w);
          }
        } else {  // pairs 8 lane + 0 .. 3 in the first chunk, 4 .. 7 in the second
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 cs = angle[r.tok][e][lane];
            float(&z)[8] = e < 2 ? u : w;
            const int b = 4 * (e & 1);
            const float z0 = z[b], z2 = z[b + 2];
            z[b] = fmaf(z0, cs.x, -z[b + 1] * cs.y);
            z[b + 1] = fmaf(z[b + 1], cs.x, z0 * cs.y);
            z[b + 2] = fmaf(z2, cs.z, -z[b + 3] * cs.w);
            z[b + 3] = fmaf(z[b + 3], cs.z, z2 * cs.w);
          }
        }
        x[i] = qkn::pack8(u);
        y[i] = qkn::pack8(w);
      }
      if (r.out != nullptr) {
        uint4* const o = reinterpret_cast<uint4*>(r.out);
        o[c0] = x[i];
        o[c1] = y[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int f = f0 + (kAhead + i) * kGroups;
      if (f < total) {
        const uint4* p = reinterpret_cast<const uint4*>(in_of(f));
        x[i] = __ldcs(p + c0);
        y[i] = __ldcs(p + c1);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& args, int num_sms, cudaStream_t stream) {
  if (args.n == 0) return cudaSuccess;
  RotaryArgs a = args;
  // Tokens of a block: what a lane group's first kAhead rows hold, so that every load goes
  // out before the angles are computed (a few rows more, in a second turn: 30.8 instead of 29.9 us for 5,033 tokens
  // of 63 rows); fewer where that would leave SMs without a block.
  const int64_t rows = a.H + a.Hk + a.Hv;
  int64_t t = kAhead * kGroups / rows;
  t = std::min<int64_t>(t, a.n / (2 * num_sms));
  a.block_tokens = (int32_t)std::max<int64_t>(1, std::min<int64_t>(t, kMaxTokens));
  rotary_kernel<<<(unsigned)((a.n + a.block_tokens - 1) / a.block_tokens), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace h3
