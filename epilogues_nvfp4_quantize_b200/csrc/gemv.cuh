// gemv_nvfp4: a few rows of bf16 or f16 activations times an NVFP4 weight (N x K).
//
//   y[m, n] = cast(G sum_k f(x[m, k]) e2m1(c[n, k]) e4m3(s[n, k / 16]) + bias[n])
//
// f is the identity or SiLU (rounded to x's type, as a separate kernel would leave it). HBM-bound:
// the weight's 9/16 byte per value is read once for up to 16 rows of x.
//
// The product runs on mma.sync.m16n8k16 (f16, float32 accumulators), weights as the 16-row operand
// and up to 8 rows of x per instruction: with so few rows tcgen05 would need the weights decoded
// into shared memory first, while here they go from a 16-byte global load through registers into
// the instruction. A weight's value without G, level x block scale, has at most 6 significant bits
// between 2^-10 and 2688 and is exact in f16. x goes to f16 by a power of two per row (the largest
// finite magnitude of the row's slice goes to [2^14, 2^15)): every bf16 value down to 2^-28 of the
// largest stays exact and smaller ones are off by at most 2^-39 of it, below float32's own sums;
// infinities and NaN stay what they are. So the arithmetic is that of float32 sums of exact
// products.
//
// A strip is 16 weight rows: rows r .. r+3 of each of the four 32-row quarters of a 128-row scale
// tile. In the tensor-core scale layout the four quarters' scales of a row are adjacent, so a strip
// reads whole 32-byte sectors. Lane (g, t) of a warp (g = lane / 4, t = lane % 4) loads 16 bytes of
// codes at columns 32 t of a 128-column group of its two rows: two whole scale blocks. The order of
// K within an instruction is free as long as both operands agree, so the lane's bytes feed the
// instructions in the order they arrive.
#pragma once

#include "ptx.cuh"
#include "codec.cuh"

namespace nvfp4 {

namespace gemvcfg {
constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr int GROUP = 128;            // columns of K per step of a warp
constexpr int TILE_TOKENS = 16;       // rows of x per pass over the weight
constexpr int ROUND = 16;             // strips between two joins of a cluster
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_SMEM = 220 * 1024;
}  // namespace gemvcfg

struct GemvArgs {
  const uint16_t* x;
  int x_f16;
  int64_t ldx;
  int64_t M, N, K;
  int silu;
  const uint8_t* codes;
  const uint8_t* sf;
  const float* gscale;
  const float* bias;
  void* D;
  int64_t ldd;
  int out_kind;          // NVFP4_OUT_*
  int kslice;            // columns of K per CTA of a cluster (a multiple of GROUP)
  int cluster;           // CTAs that share K
  int kwarps;            // warps that share a CTA's slice (a power of two)
  int64_t strips;
};

__host__ __device__ constexpr int gemv_x_pitch(int kslice) { return kslice * 2 + 64; }  // bytes per row of x
__host__ __device__ constexpr int gemv_smem(int nt, int kslice, int cluster) {
  return 8 * nt * gemv_x_pitch(kslice) + 2 * gemvcfg::WARPS * 512 * nt + (cluster > 1 ? gemvcfg::ROUND * 512 * nt : 0) +
         8 * nt * 4 + 64 * 4;
}

__device__ __forceinline__ float gemv_act(float v, int silu) {
  return silu ? v / (1.0f + expf(-v)) : v;
}

__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.u8.u32 c, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// One step's codes and scales of a lane: 32 columns of rows n0 and n1.
struct GemvStep {
  uint4 c[2];
  uint32_t s[2];  // two E4M3 codes each
};

template <int NT>
__global__ void __launch_bounds__(gemvcfg::THREADS, 1) gemv_nvfp4_kernel(const GemvArgs a) {
  using namespace gemvcfg;
  extern __shared__ __align__(128) uint8_t gemv_smem_raw[];
  const int pitch = gemv_x_pitch(a.kslice);
  uint8_t* xs = gemv_smem_raw;
  float* red = reinterpret_cast<float*>(xs + 8 * NT * pitch);   // [2][WARPS][32][4 NT]
  float* part = red + 2 * WARPS * 128 * NT;                      // [ROUND][32][4 NT] (clusters)
  float* inv = part + (a.cluster > 1 ? ROUND * 128 * NT : 0);    // factor of each row of x
  unsigned* amax = reinterpret_cast<unsigned*>(inv + 8 * NT);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % a.cluster;
  const int64_t cid = blockIdx.x / a.cluster, ncluster = gridDim.x / a.cluster;
  const int64_t k0 = static_cast<int64_t>(rank) * a.kslice;
  const int64_t kleft = a.K - k0;
  const int klen = static_cast<int>(kleft < 0 ? 0 : kleft < a.kslice ? kleft : a.kslice);  // a multiple of 64
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
  const int tokens = static_cast<int>(a.M - m0 < 8 * NT ? a.M - m0 : 8 * NT);

  // ---- this slice of x into shared memory as f16, each row by its power of two ----------
  if (tid < 8 * NT) amax[tid] = 0u;
  __syncthreads();
  const int vecs = klen >> 3;
  auto load_x = [&](int m, int v, float (&f)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.x + (m0 + m) * a.ldx + k0 + 8 * v));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (a.x_f16) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
      } else {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
    }
    if (a.silu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = gemv_act(f[i], 1);
        f[i] = a.x_f16 ? __half2float(__float2half_rn(f[i])) : __bfloat162float(__float2bfloat16_rn(f[i]));
      }
    }
  };
  // Pass 1: the largest finite magnitude of each row (a row has a multiple of 8 vectors, so the
  // eight lanes of an octet share a row). Pass 2 reads the slice again from L2.
  for (int i = tid; i < tokens * vecs; i += THREADS) {
    const int m = i / vecs;
    float f[8], big = 0.0f;
    load_x(m, i - m * vecs, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float z = fabsf(f[k]);
      if (z <= 3.4028234663852886e38f) big = fmaxf(big, z);
    }
    const uint32_t octet = 0xFFu << (lane & 24);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(octet, big, o));
    if ((lane & 7) == 0) atomicMax(amax + m, __float_as_uint(big));
  }
  __syncthreads();
  const int xvecs = a.kslice / 8;
  for (int i = tid; i < 8 * NT * xvecs; i += THREADS) {
    const int m = i / xvecs, v = i - m * xvecs;
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (m < tokens) {
      // the row's factor 2^(14 - e) and its inverse; the clamp keeps both normal float32 numbers
      int e = static_cast<int>(amax[m] >> 23) - 127;
      if (e < -100) e = -100;
      if (v == 0) inv[m] = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
      if (v < vecs) {
        const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
        float f[8];
        load_x(m, v, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= up;
        o = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
      }
    } else if (v == 0) {
      inv[m] = 0.0f;
    }
    // columns 32 t + 8 w .. + 7 of a group sit at 64 w + 16 t bytes of it
    *reinterpret_cast<uint4*>(xs + m * pitch + (v >> 4) * 256 + (v & 3) * 64 + ((v >> 2) & 3) * 16) = o;
  }
  __syncthreads();

  // ---- strips ---------------------------------------------------------------------------
  const int wk = warp & (a.kwarps - 1), wr = warp / a.kwarps, rows_at_once = WARPS / a.kwarps;
  const int groups = a.kslice / GROUP;
  const int per = (groups + a.kwarps - 1) / a.kwarps;
  const int gb = wk * per, ge = gb + per < groups ? gb + per : groups;  // this warp's groups of the slice
  const float G = *a.gscale;
  const int64_t kgroups64 = a.K >> 6;

  auto load_step = [&](int64_t tile, int r, int64_t n0, int grp, GemvStep& st) {
    const int64_t k = k0 + static_cast<int64_t>(grp) * GROUP + 32 * t;
    st.c[0] = st.c[1] = make_uint4(0u, 0u, 0u, 0u);
    st.s[0] = st.s[1] = 0u;
    if (k < a.K) {
      const uint8_t* sp = a.sf + (tile * kgroups64 + (k >> 6)) * 512 + (r * 4 + (g >> 2)) * 4 + ((k >> 4) & 3);
      const uint8_t* cp = a.codes + n0 * (a.K >> 1) + (k >> 1);
      if (n0 < a.N) {
        st.c[0] = __ldg(reinterpret_cast<const uint4*>(cp));
        st.s[0] = __ldg(reinterpret_cast<const uint16_t*>(sp));
      }
      if (n0 + 64 < a.N) {
        st.c[1] = __ldg(reinterpret_cast<const uint4*>(cp + 64 * (a.K >> 1)));
        st.s[1] = __ldg(reinterpret_cast<const uint16_t*>(sp + 8));
      }
    }
  };
  float acc[NT][4];
  auto compute = [&](int grp, const GemvStep& st) {
    uint32_t s2[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(st.s[i])));
      s2[i][0] = __byte_perm(h2, h2, 0x1010);
      s2[i][1] = __byte_perm(h2, h2, 0x3232);
    }
    const uint32_t c0[4] = {st.c[0].x, st.c[0].y, st.c[0].z, st.c[0].w};
    const uint32_t c1[4] = {st.c[1].x, st.c[1].y, st.c[1].z, st.c[1].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0[4], a1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a0[j] = mul_f16x2(e2m1x2_to_f16x2((c0[w] >> (8 * j)) & 0xFFu), s2[0][w >> 1]);
        a1[j] = mul_f16x2(e2m1x2_to_f16x2((c1[w] >> (8 * j)) & 0xFFu), s2[1][w >> 1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 xb = *reinterpret_cast<const uint4*>(xs + (8 * n + g) * pitch + grp * 256 + w * 64 + t * 16);
        mma_16x8x16(acc[n], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
        mma_16x8x16(acc[n], a0[2], a1[2], a0[3], a1[3], xb.z, xb.w);
      }
    }
  };
  // value i of lane's fragment: weight row g or g + 8 of the strip, row 2 t or 2 t + 1 of x
  auto put = [&](int64_t strip, int n, int i, float v) {
    const int m = 8 * n + 2 * t + (i & 1);
    const int64_t row = (strip >> 3) * 128 + (g >> 2) * 32 + (i >> 1) * 64 + (strip & 7) * 4 + (g & 3);
    if (m >= tokens || row >= a.N) return;
    if (a.bias != nullptr) v += a.bias[row];
    const int64_t at = (m0 + m) * a.ldd + row;
    if (a.out_kind == 2) {
      static_cast<float*>(a.D)[at] = v;
    } else if (a.out_kind == 1) {
      static_cast<__half*>(a.D)[at] = __float2half_rn(v);
    } else {
      static_cast<__nv_bfloat16*>(a.D)[at] = __float2bfloat16_rn(v);
    }
  };

  const int64_t per_iter = ncluster * rows_at_once;
  const int64_t iters = (a.strips + per_iter - 1) / per_iter;
  int buf = 0, in_round = 0;
  int64_t round_base = 0;  // first iteration of the round
  for (int64_t it = 0; it < iters; ++it) {
    const int64_t strip = it * per_iter + cid * rows_at_once + wr;
    const bool have = strip < a.strips;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    if (have) {
      const int64_t tile = strip >> 3;
      const int r = static_cast<int>(strip & 7) * 4 + (g & 3);
      const int64_t n0 = tile * 128 + (g >> 2) * 32 + r;
      for (int grp = gb; grp < ge; ++grp) {
        GemvStep st;
        load_step(tile, r, n0, grp, st);
        compute(grp, st);
      }
    }
    float* mine = red + ((buf * WARPS + warp) * 32 + lane) * 4 * NT;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[4 * n + i] = acc[n][i];
    __syncthreads();
    // the warps of a strip take turns at adding up its pieces of K
    if (wk == static_cast<int>(it) % a.kwarps && have) {
      float sum[4 * NT];
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) sum[i] = 0.0f;
      for (int w = 0; w < a.kwarps; ++w) {
        const float* p = red + ((buf * WARPS + wr * a.kwarps + w) * 32 + lane) * 4 * NT;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) sum[i] += p[i];
      }
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) sum[i] = sum[i] * G * inv[8 * (i >> 2) + 2 * t + (i & 1)];
      if (a.cluster == 1) {
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) put(strip, i >> 2, i & 3, sum[i]);
      } else {
        float* p = part + ((in_round + wr) * 32 + lane) * 4 * NT;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) p[i] = sum[i];
      }
    }
    buf ^= 1;
    if (a.cluster > 1) {
      in_round += rows_at_once;
      if (in_round + rows_at_once > ROUND || it == iters - 1) {
        cluster_sync_all();  // every CTA's pieces of this round's strips are written
        const int have_slots = in_round;
        for (int s = rank + a.cluster * warp; s < have_slots; s += a.cluster * WARPS) {
          const int64_t sit = round_base + s / rows_at_once;
          const int64_t st = sit * per_iter + cid * rows_at_once + s % rows_at_once;
          if (st >= a.strips) continue;
          const uint32_t at = smem_u32(part + (s * 32 + lane) * 4 * NT);
          float sum[4 * NT];
#pragma unroll
          for (int i = 0; i < 4 * NT; ++i) sum[i] = 0.0f;
          for (int c = 0; c < a.cluster; ++c) {
            const uint32_t remote = mapa_shared(at, c);
#pragma unroll
            for (int i = 0; i < 4 * NT; ++i) sum[i] += ld_cluster_f32(remote + 4 * i);
          }
#pragma unroll
          for (int i = 0; i < 4 * NT; ++i) put(st, i >> 2, i & 3, sum[i]);
        }
        cluster_sync_all();  // no CTA overwrites or leaves before the others have read
        in_round = 0;
        round_base = it + 1;
      }
    }
  }
}

}  // namespace nvfp4
