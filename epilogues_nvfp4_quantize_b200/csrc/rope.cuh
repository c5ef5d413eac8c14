// rope_axes: rotary positions with one to four axes (time, height, width) on heads of Q and K.
//
// Pair p of a head belongs to one axis a(p) and has a frequency f_p. With the row's position
// t_a on that axis, the pair (u, v) becomes (u cos A - v sin A, u sin A + v cos A),
// A = t_a(p) f_p; the inverse (and the gradient) is the same with -A. HBM-bound: every element is
// read and written once (plus the positions).
//
// Angles: A grows with the position while only A mod 2 pi matters, so t f and its reduction are
// in float64 (a float32 product at t = 10^6 is off by 0.06 rad); the reduced angle, at most pi,
// goes to sincospif in float32 (error about 2e-7). All heads of a row share its angles, so a CTA
// computes them once into shared memory and then walks its rows' heads with 16-byte accesses.
#pragma once

#include "ptx.cuh"
#include "codec.cuh"
#include "quantize.cuh"

namespace nvfp4 {

namespace ropecfg {
constexpr int THREADS = 256;
// Heads in flight per thread (of 2, 4, 6 and 8, with the best rows per CTA for each: 23.0, 21.8, 21.7,
// 22.7 us on 4096 x 24 x 256 in bf16); half as many where a head takes two accesses.
constexpr int BATCH = 6, BATCH_HALVES = 3;
constexpr int MAX_AXES = 4;
constexpr int MAX_HEAD_DIM = 1024;
constexpr int MAX_TABLE_BYTES = 16384;  // cos/sin pairs of a CTA's rows
}  // namespace ropecfg

enum RopeMode { ROPE_INTERLEAVED = 0, ROPE_HALVES = 1, ROPE_HALVES_SCALAR = 2 };

struct RopeArgs {
  const void* x;
  void* y;
  int64_t rows;
  int heads, head_dim;
  int64_t x_row, x_head, y_row, y_head;  // strides in elements
  const void* pos;
  int pos_f32;                           // positions are float32 (else int32)
  int64_t ldpos;
  const double* freqs;                   // npairs, in radians per position
  int npairs;                            // rotated pairs; elements past 2 * npairs pass through
  int axis_end[ropecfg::MAX_AXES];       // axis a holds pairs [axis_end[a-1], axis_end[a])
  int inverse;
  int rows_per_cta;
  int in_place;                          // y is x: what passes through stays where it is
  int table_pitch;                       // pairs per row of the table (npairs to the next multiple of 4)
  int units, slots;                      // pieces of a head, and how many heads the CTA takes at once
  int step_rows, step_heads;             // `slots` heads further on
  float inv_units, inv_heads, inv_pairs; // for quotients of small numbers
};

// a / b for 0 <= a < 2^15 and 0 < b < 2^15, with inv_b = 1 / b: the float32 error is below 2^-7 / b, and
// a + 1/2 keeps the quotient 1 / (2 b) away from the next whole number.
__device__ __forceinline__ int small_quotient(int a, float inv_b) {
  return static_cast<int>((static_cast<float>(a) + 0.5f) * inv_b);
}

template <class T>
struct RopeVec;  // 16 bytes of T as floats
template <>
struct RopeVec<float> {
  static constexpr int V = 4;
  __device__ static void unpack(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
  }
  __device__ static uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int V = 8;
  __device__ static void unpack(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  __device__ static uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct RopeVec<__half> {
  static constexpr int V = 8;
  __device__ static void unpack(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ static uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                      pack_f16x2(v[6], v[7]));
  }
};

__device__ __forceinline__ float rope_f32(float v) { return v; }
__device__ __forceinline__ float rope_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float rope_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void rope_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void rope_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void rope_put(__half* p, float v) { *p = __float2half_rn(v); }

// cos and sin of the pairs of this CTA's rows, in two tables (a thread reads those of four pairs at a
// time: interleaved with one another, they conflicted in shared memory's banks).
__device__ __forceinline__ void rope_table(const RopeArgs& a, int64_t row0, int nrows, float* cosines, float* sines) {
  for (int i = threadIdx.x; i < nrows * a.npairs; i += ropecfg::THREADS) {
    const int r = small_quotient(i, a.inv_pairs), p = i - r * a.npairs;
    int ax = 0;
#pragma unroll
    for (int k = 0; k < ropecfg::MAX_AXES - 1; ++k) ax += p >= a.axis_end[k] ? 1 : 0;
    const int64_t at = (row0 + r) * a.ldpos + ax;
    const double t = a.pos_f32 ? static_cast<double>(static_cast<const float*>(a.pos)[at])
                               : static_cast<double>(static_cast<const int*>(a.pos)[at]);
    double u = t * a.freqs[p] * 0.31830988618379067154;  // in units of pi
    u -= 2.0 * rint(0.5 * u);
    float s, c;
    sincospif(static_cast<float>(u), &s, &c);
    cosines[r * a.table_pitch + p] = c;
    sines[r * a.table_pitch + p] = a.inverse ? -s : s;
  }
}

// A unit is what one thread does to one head: 16 bytes (interleaved pairs), two times 16 bytes
// (the same places of both halves) or a 16-byte piece that passes through, and with
// ROPE_HALVES_SCALAR (a number of pairs that 16 bytes do not divide) one pair or one element.
// Threads keep their unit and walk the (row, head) pairs of the CTA, a batch at a time. A CTA's first
// batch is loaded before its table is made, so the positions, the angles and x travel together.
template <class T, int MODE>
__global__ void __launch_bounds__(ropecfg::THREADS, MODE == ROPE_HALVES ? 3 : 4) rope_kernel(const RopeArgs a) {
  using namespace ropecfg;
  using RV = RopeVec<T>;
  constexpr int V = RV::V;
  extern __shared__ float rope_cos[];
  float* const rope_sin = rope_cos + a.rows_per_cta * a.table_pitch;
  constexpr int B = MODE == ROPE_HALVES ? BATCH_HALVES : BATCH;
  constexpr int NP = MODE == ROPE_INTERLEAVED ? V / 2 : V;  // pairs of a unit
  griddep_launch_dependents();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_cta;
  const int nrows = static_cast<int>(a.rows - row0 < a.rows_per_cta ? a.rows - row0 : a.rows_per_cta);
  const int n = a.npairs, units = a.units, slots = a.slots;
  const int slot = slots > 1 ? small_quotient(threadIdx.x, a.inv_units) : 0;
  const int total = nrows * a.heads;
  // Row and head of this thread's first step, then `slots` heads further each time; offsets are moved
  // along instead of multiplied out.
  const int r_first = small_quotient(slot, a.inv_heads), h_first = slot - r_first * a.heads;
  struct Place {
    int r, h;
    int64_t at;  // element of x or y
  };
  auto first = [&](int64_t row, int64_t head) { return Place{r_first, h_first, r_first * row + h_first * head}; };
  const int64_t x_step = a.step_rows * a.x_row + a.step_heads * a.x_head, x_wrap = a.x_row - a.heads * a.x_head;
  const int64_t y_step = a.step_rows * a.y_row + a.step_heads * a.y_head, y_wrap = a.y_row - a.heads * a.y_head;
  auto advance = [&](Place& p, int64_t step, int64_t wrap) {
    p.r += a.step_rows;
    p.h += a.step_heads;
    p.at += step;
    if (p.h >= a.heads) {
      p.h -= a.heads;
      ++p.r;
      p.at += wrap;
    }
  };
  const T* const x = static_cast<const T*>(a.x) + row0 * a.x_row;
  T* const y = static_cast<T*>(a.y) + row0 * a.y_row;
  int u = threadIdx.x - slot * units;
  bool rotates;
  int e0;  // first element of the unit within the head
  auto unit = [&]() {
    rotates = MODE == ROPE_INTERLEAVED ? u * (V / 2) < n : MODE == ROPE_HALVES ? u * V < n : u < n;
    e0 = MODE == ROPE_INTERLEAVED ? u * V
         : MODE == ROPE_HALVES    ? (rotates ? u * V : 2 * n + (u - n / V) * V)
                                  : (rotates ? u : n + u);
  };
  unit();
  const bool works = slot < slots && u < units;
  uint4 lo[B], hi[B];
  Place from = first(a.x_row, a.x_head);
  auto load = [&](int j) {
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (j + k * slots < total) {
        const T* src = x + from.at + e0;
        lo[k] = *reinterpret_cast<const uint4*>(src);
        if (MODE == ROPE_HALVES && rotates) hi[k] = *reinterpret_cast<const uint4*>(src + n);
      }
      advance(from, x_step, x_wrap);
    }
  };
  griddep_wait();  // nothing before this reads or writes global memory
  if (MODE != ROPE_HALVES_SCALAR && works && (rotates || !a.in_place)) load(slot);
  rope_table(a, row0, nrows, rope_cos, rope_sin);
  __syncthreads();
  if (!works) return;

  for (; u < units; u += THREADS) {  // once, unless a head has more units than the CTA threads
    unit();
    if (!rotates && a.in_place) continue;
    // the pairs' cos and sin stay in registers while the row is the same
    float c[NP], sn[NP];
    const bool whole = (u + 1) * NP <= n;  // else the unit's last pairs pass through
    Place to = first(a.y_row, a.y_head);
    int of = -1;
    if (u >= THREADS || MODE == ROPE_HALVES_SCALAR) from = first(a.x_row, a.x_head);
    for (int j = slot; j < total; j += B * slots) {
      if constexpr (MODE != ROPE_HALVES_SCALAR) {
        if (j != slot || u >= THREADS) load(j);
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (j + k * slots < total) {
          T* const dst = y + to.at + e0;
          const int r = to.r;
          if constexpr (MODE == ROPE_HALVES_SCALAR) {
            const T* const src = x + from.at + e0;
            if (!rotates) {
              *dst = *src;
            } else {
              const float p = rope_f32(src[0]), q = rope_f32(src[n]);
              const float c1 = rope_cos[r * a.table_pitch + u], s1 = rope_sin[r * a.table_pitch + u];
              rope_put(dst, p * c1 - q * s1);
              rope_put(dst + n, p * s1 + q * c1);
            }
          } else {
            if (rotates) {
              if (r != of) {
                of = r;
                const float* const ct = rope_cos + r * a.table_pitch + u * NP;
                const float* const st = rope_sin + r * a.table_pitch + u * NP;
                if constexpr (NP % 4 == 0) {
#pragma unroll
                  for (int i = 0; i < NP; i += 4) {
                    const float4 c4 = *reinterpret_cast<const float4*>(ct + i), s4 = *reinterpret_cast<const float4*>(st + i);
                    c[i] = c4.x, c[i + 1] = c4.y, c[i + 2] = c4.z, c[i + 3] = c4.w;
                    sn[i] = s4.x, sn[i + 1] = s4.y, sn[i + 2] = s4.z, sn[i + 3] = s4.w;
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < NP; ++i) c[i] = ct[i], sn[i] = st[i];
                }
              }
              float v[V];
              RV::unpack(lo[k], v);
              if constexpr (MODE == ROPE_INTERLEAVED) {
                auto turn = [&](int i) {
                  const float s0 = v[2 * i], s1 = v[2 * i + 1];
                  v[2 * i] = s0 * c[i] - s1 * sn[i];
                  v[2 * i + 1] = s0 * sn[i] + s1 * c[i];
                };
                if (whole) {
#pragma unroll
                  for (int i = 0; i < NP; ++i) turn(i);
                } else {
#pragma unroll
                  for (int i = 0; i < NP; ++i) {
                    if (u * NP + i < n) turn(i);
                  }
                }
              } else {
                float w[V];
                RV::unpack(hi[k], w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                  const float s0 = v[i], s1 = w[i];
                  v[i] = s0 * c[i] - s1 * sn[i];
                  w[i] = s0 * sn[i] + s1 * c[i];
                }
                *reinterpret_cast<uint4*>(dst + n) = RV::pack(w);
              }
              lo[k] = RV::pack(v);
            }
            *reinterpret_cast<uint4*>(dst) = lo[k];
          }
        }
        advance(to, y_step, y_wrap);
        if constexpr (MODE == ROPE_HALVES_SCALAR) advance(from, x_step, x_wrap);
      }
    }
  }
}

}  // namespace nvfp4
