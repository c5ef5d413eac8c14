// gemv_nvfp4: a few rows of bf16 or f16 activations times an NVFP4 weight (N x K).
//
//   y[m, n] = cast(G sum_k f(x[m, k]) e2m1(c[n, k]) e4m3(s[n, k / 16]) + bias[n])
//
// f is the identity or SiLU. HBM-bound: the weight's 9/16 byte per value is read once for up to 16 rows
// of x.
//
// The product runs on mma.sync.m16n8k16 (f16, float32 accumulators), weights as the 16-row operand
// and up to 8 rows of x per instruction: with so few rows tcgen05 would need the weights decoded
// into shared memory first, while here they go from shared memory through registers into the
// instruction. A weight's value without G, level x block scale, has at most 6 significant bits
// between 2^-10 and 2688 and is exact in f16. x goes to f16 by a power of two for each 128 columns of a
// row (their largest finite magnitude goes to [2^14, 2^15)): every bf16 value down to 2^-28 of that
// stays exact and smaller ones are off by at most 2^-39 of it, below float32's own sums; infinities and
// NaN stay what they are. So the arithmetic is that of float32 sums of exact products. SiLU's values, which
// have float32's digits, are each a sum of two f16 (2^-22 of the value, or the 2^-39 above), and both go
// through the tensor core with the same weights. (Rounded to one f16, an output in float32 was off by 2^-11 of
// a product and one in f16 by as much again as its own rounding. Up to four rows of x the second part is free,
// with more it takes a fifth of the time: 8 x 4096 x 24576 18.5 -> 22.3 us, 16 rows 25.0 -> 31.7.)
//
// A strip is 16 weight rows: rows r .. r+3 of each of the four 32-row quarters of a 128-row scale
// tile. In the tensor-core scale layout the four quarters' scales of a row are adjacent, so a strip
// reads whole 32-byte sectors. Lane (g, t) of a warp (g = lane / 4, t = lane % 4) takes 16 bytes of
// codes at columns 32 t of a 128-column group of its two rows: two whole scale blocks. The order of
// K within an instruction is free as long as both operands agree, so the lane's bytes feed the
// instructions in the order they come.
//
// Measured: 2 x 4096 x 98304 runs at 5.0 TB/s (45 us); of 2 x 4096 x 24576's 16.7 us, 8.7 are the bytes at the
// copy rate and about 5 the start (x to every SM and to f16 there, the first weights).
#pragma once

#include "ptx.cuh"
#include "codec.cuh"
#include "quantize.cuh"

namespace nvfp4 {

namespace gemvcfg {
constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr int GROUP = 128;            // columns of K per step of a warp
constexpr int ROUND = 16;             // strips between two joins of a cluster
constexpr int STEPS = 2;              // steps whose weights are copied together, a chunk
constexpr int CODES = 16 * STEPS * GROUP / 2, CHUNK = CODES + STEPS * 128;  // bytes of its codes; with its scales
constexpr int PAIR_TOKENS = 2;        // rows of x up to which block scales multiply sums instead of weights
constexpr int ZEROS = 256;            // bytes of 0 in shared memory, for that
constexpr int MAX_SMEM = 220 * 1024;
}  // namespace gemvcfg

// The eight columns of the instruction: rows of x; two of them for each lane t; four for each half of t.
enum GemvPair { PAIR_NO = 0, PAIR_LANES = 1, PAIR_HALVES = 2 };
enum GemvSilu { SILU_NO = 0, SILU_ROWS = 1, SILU_PARTS = 2 };

struct GemvArgs {
  const uint16_t* x;
  int x_f16;
  int64_t ldx;
  int64_t M, N, K;
  int tile;              // rows of x per CTA
  const uint8_t* codes;
  const uint8_t* sf;
  const float* gscale;
  const float* bias;
  void* D;
  int64_t ldd;
  int out_kind;          // NVFP4_OUT_*
  int kslice;            // columns of K per CTA of a cluster (a multiple of GROUP)
  int cluster_log2;      // log2 of the CTAs that share K
  int kwarps_log2;       // log2 of the warps that share a CTA's slice
  int per;               // steps of each of those warps
  int strips;
  int strips_at_once;    // of the whole grid
  int iters;             // strips each warp takes
};

__host__ __device__ constexpr int gemv_x_pitch(int kslice) { return kslice * 2 + 64; }  // bytes per row of x
// Bytes from the first f16 of a value to the second: like neighbouring rows, the two lie in different halves of
// the 32 banks.
__host__ __device__ constexpr int gemv_x_rest(int tokens, int kslice) {
  return tokens * gemv_x_pitch(kslice) + (tokens & 1 ? 0 : 64);
}
// `tokens`: rows of x per CTA; `parts`: f16 values for each of theirs.
__host__ __device__ constexpr int gemv_smem(int nt, int buffers, int tokens, int parts, int kslice, int cluster) {
  return gemvcfg::WARPS * buffers * gemvcfg::CHUNK +                                             // ring of weights
         2 * gemvcfg::WARPS * 512 * nt + (cluster > 1 ? 2 * gemvcfg::ROUND * 512 * nt : 0) +     // joins
         kslice / gemvcfg::GROUP * 8 * nt * 4 +                                                  // factors of x
         parts * gemv_x_rest(tokens, kslice) +                                                   // x
         (tokens <= gemvcfg::PAIR_TOKENS ? gemvcfg::ZEROS : 0);
}

__device__ __forceinline__ void gemv_unpack(const uint4& q, int f16, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (f16) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    } else {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

// x / (1 + e^-x), within 2^-21 of the value (expf 2^-22, the sum, the reciprocal and the product one
// float32 step together); where 1 + e^-x passes 2^126 and the value is below 2^-119, 0.
__device__ __forceinline__ float gemv_silu(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-x)));
  return x * r;
}

// Largest finite magnitude of eight 16-bit floats: without their signs they compare like integers, two
// at a time; where infinities or NaN come out on top, they are left out one by one.
__device__ __forceinline__ float gemv_finite_amax(const uint4& q, int f16) {
  const uint32_t w[4] = {q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu, q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu};
  const uint32_t m2 = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  const uint32_t inf = f16 ? 0x7C00u : 0x7F80u;
  if (m >= inf) {
    m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
      m = max(m, max(lo < inf ? lo : 0u, hi < inf ? hi : 0u));
    }
  }
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(m))) : __uint_as_float(m << 16);
}

// Eight E2M1 codes to four f16 pairs, in their order. Taking the bytes apart inside the PTX costs
// about one instruction per pair; shifting and masking them out first was measured at four.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t c, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(c));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Lanes 8 i .. 8 i + 7 give the addresses of 16-byte rows; lane (g, t) gets word t of row g of each i.
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16x8x16_from0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Barrier of `threads` threads, by its id (0 is __syncthreads).
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Asynchronous copy to shared memory; bytes past `n` of the 16 are written as 0.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_async16_hint(uint32_t dst, const void* src, int n, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// BUFFERS (a power of two): chunks of weights in flight per warp.
// PAIR: at most two rows of x; PAIR_HALVES two with SiLU, PAIR_LANES otherwise.
// SILU: f is SiLU, whose values are sums of two f16, the second ones `x_rest` bytes behind the first. As long as
// the instruction's eight columns have room (SILU_ROWS: four rows of x, with PAIR one) the two are columns next to
// one another, which costs the products nothing; above that they are read one after the other (SILU_PARTS).
template <int NT, int BUFFERS, int PAIR, int SILU>
__global__ void __launch_bounds__(gemvcfg::THREADS, 1) gemv_nvfp4_kernel(const GemvArgs a) {
  using namespace gemvcfg;
  extern __shared__ __align__(128) uint8_t gemv_smem_raw[];
  const int cluster = 1 << a.cluster_log2, kwarps = 1 << a.kwarps_log2;
  const int pitch = gemv_x_pitch(a.kslice);
  uint8_t* ring = gemv_smem_raw;                                               // [WARPS][BUFFERS][CHUNK]
  float* red = reinterpret_cast<float*>(ring + WARPS * BUFFERS * CHUNK);       // [2][WARPS][32][4 NT]
  float* part = red + 2 * WARPS * 128 * NT;                                    // [2][ROUND][32][4 NT] (clusters)
  float* inv = part + (cluster > 1 ? 2 * ROUND * 128 * NT : 0);                // [groups][8 NT] factors of x
  uint8_t* xs = reinterpret_cast<uint8_t*>(inv + a.kslice / GROUP * 8 * NT);   // [tokens][pitch]

  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) & (cluster - 1);
  const int cid = static_cast<int>(blockIdx.x) >> a.cluster_log2;
  const int k0 = rank * a.kslice;
  const int kleft = static_cast<int>(a.K) - k0;
  const int klen = kleft < 0 ? 0 : kleft < a.kslice ? kleft : a.kslice;  // a multiple of 64
  const int64_t m0 = (static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * a.tile;
  if (m0 >= a.M) return;  // the whole cluster
  const int tokens = static_cast<int>(a.M - m0 < a.tile ? a.M - m0 : a.tile);
  if (cluster > 1) cluster_arrive();
  const int x_rest = gemv_x_rest(tokens, a.kslice);

  // ---- this slice of x on its way into shared memory -------------------------------------
  // Columns 32 t + 8 w .. + 7 of a group sit at 64 w + 16 t bytes of it (PAIR_HALVES: columns in order). Each row
  // is taken by as many warps as there are (one at least); a half-warp takes a whole group.
  const int vecs = klen >> 3, xvecs = a.kslice >> 3;
  const int xwarps_log2 = tokens <= 1 ? 4 : tokens <= 2 ? 3 : tokens <= 4 ? 2 : tokens <= 8 ? 1 : 0;
  const int xm = warp >> xwarps_log2;
  auto each_vector = [&](auto&& body) {
    if (xm >= tokens) return;
    uint8_t* row = xs + xm * pitch;
    for (int v = ((warp & ((1 << xwarps_log2) - 1)) << 5) + lane; v < xvecs; v += 32 << xwarps_log2)
      body(v, reinterpret_cast<uint4*>(row + (PAIR == PAIR_HALVES ? v * 16 : (v >> 4) * 256 + (v & 3) * 64 + ((v >> 2) & 3) * 16)));
  };
  griddep_wait();  // nothing before this reads or writes global memory
  {
    const uint16_t* row = a.x + (m0 + xm) * a.ldx + k0;
    each_vector([&](int v, uint4* p) { copy_async16(smem_u32(p), v < vecs ? row + 8 * v : a.x, v < vecs ? 16 : 0); });
  }
  copy_async_commit();
  const float G = *a.gscale;

  // ---- the walk over weights: step = one 128-column group of one strip ---------------------
  // Every warp takes `per` groups of each of its strips (groups past the slice are skipped), so the
  // warps of a strip reach its join together. A warp copies its weights in chunks of STEPS groups: eight
  // lanes a row, so an instruction covers four rows of the strip (those of one quarter) in whole lines.
  // The second half of every other row comes first, so that the eight lanes of an access, four of
  // each of two rows, find different banks.
  // (Copied by the lane that uses them, 64 bytes a row and 4 bytes of scales at a time, so that nothing else
  // had to be waited for, they took 35 instructions per step instead of 16. Bulk copies of 256 bytes a
  // row are limited by the number of copies, 17 cycles each: 98304 rows of 4096 in 57 us.)
  const int wk = warp & (kwarps - 1), wr = warp >> a.kwarps_log2, rows_at_once = WARPS >> a.kwarps_log2;
  const int groups = (klen + GROUP - 1) / GROUP;
  const int gb = wk * a.per;
  const int my_groups = groups - gb < a.per ? groups - gb : a.per;     // of each strip; may be 0 or less
  const int chunks = (a.per + STEPS - 1) / STEPS;
  const int left = klen - gb * GROUP < a.per * GROUP ? klen - gb * GROUP : a.per * GROUP;  // columns of each strip
  const int64_t krow = a.K >> 1;  // bytes of codes per weight row

  // The next chunk to load. Rows past N and columns past the slice become 0.
  int l_strip = cid * rows_at_once + wr;
  int l_chunk = 0;
  int l_rows;                    // from the lane's row of quarter 0 to N
  const uint8_t *l_codes, *l_sf;  // the lane's 16 bytes of quarter 0; of the scales (row lane & 3 of unit lane / 4)
  auto seek = [&]() {
    const int64_t s = l_strip < a.strips ? l_strip : a.strips - 1;
    const int64_t tile = s >> 3;
    const int r = static_cast<int>(s & 7) * 4;
    const int64_t n = tile * 128 + r + (lane >> 3), k = k0 + gb * GROUP;
    l_rows = static_cast<int>(a.N - n < 128 ? a.N - n : 128);
    l_codes = a.codes + n * krow + (k >> 1) + (lane & 7) * 16;
    l_sf = a.sf + (tile * (a.K >> 6) + (k >> 6) + (lane >> 2)) * 512 + (r + (lane & 3)) * 16;
  };
  // codes are read once per call: they leave L2 first, so that x and what else is used again stay
  const uint64_t once = l2_policy_evict_first();
  const uint32_t my_ring = smem_u32(ring) + warp * (BUFFERS * CHUNK);
  // PAIR_HALVES reads eight rows of 16 bytes at a time: there the 16-byte piece c of row r goes to c ^ (r & 7).
  const uint32_t put_at = PAIR == PAIR_HALVES ? (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 3)) * 16
                                              : (lane >> 3) * 128 + (((lane & 7) * 16) ^ ((lane & 8) << 3));
  const uint32_t put_odd = PAIR == PAIR_HALVES ? put_at ^ 64 : put_at;  // of quarters 1 and 3: rows 4 to 7 of eight
  auto load = [&](int b) {
    if (l_strip < a.strips) {
      const int cols = left - l_chunk * (STEPS * GROUP);
      const uint32_t dst = my_ring + b * CHUNK;
      const int rows = (lane & 7) * 32 < cols ? l_rows : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        copy_async16_hint(dst + q * 512 + (q & 1 ? put_odd : put_at), rows > 32 * q ? l_codes + q * 32 * krow : a.codes, rows > 32 * q ? 16 : 0, once);
      if (lane < 8 * STEPS) {
        const bool in = (lane >> 2) * 64 < cols;
        copy_async16(dst + CODES + lane * 16, in ? l_sf : a.sf, in ? 16 : 0);
      }
      l_codes += STEPS * (GROUP / 2);
      l_sf += STEPS * 1024;
      if (++l_chunk == chunks) {
        l_chunk = 0;
        l_strip += a.strips_at_once;
        seek();
      }
    }
    copy_async_commit();
  };
  seek();
#pragma unroll
  for (int b = 0; b < BUFFERS; ++b) load(b);

  // ---- x to f16, each 128 columns of a row by their power of two -------------------------
  // The largest finite magnitude of a group goes to [2^14, 2^15). A half-warp holds the group, so
  // nothing has to be known of the rest of the row, and the products of a group are scaled back when
  // they are added to the others.
  copy_async_wait<BUFFERS>();
  if (!SILU && a.x_f16) {  // f16 needs no factor
    for (int i = tid; i < a.kslice / GROUP * 8 * NT; i += THREADS) inv[i] = 1.0f;
  } else {
    each_vector([&](int v, uint4* p) {
      uint4 q = *p;
      float f[8];
      gemv_unpack(q, a.x_f16, f);
      if constexpr (SILU) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = gemv_silu(f[k]);
        // for the largest magnitude only: a value that rounds up a power of two still fits f16
        q = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      }
      float big = gemv_finite_amax(q, !SILU && a.x_f16);
      const uint32_t half = 0xFFFFu << (lane & 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(half, big, o));
      // 2^(14 - e) and its inverse; the clamp keeps both normal float32 numbers (a bf16 value is a multiple of
      // 2^-133, so below it all of them are exact in f16 all the same)
      int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
      if (e < -112) e = -112;
      const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      if ((lane & 15) == 0) {
        const float down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
        if constexpr (SILU == SILU_ROWS) {
          *reinterpret_cast<float2*>(inv + (v >> 4) * 8 * NT + 2 * xm) = make_float2(down, down);
        } else {
          inv[(v >> 4) * 8 * NT + xm] = down;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= up;
      const uint32_t h[4] = {pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7])};
      *p = make_uint4(h[0], h[1], h[2], h[3]);
      if constexpr (SILU) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __half2 h2 = *reinterpret_cast<const __half2*>(&h[k >> 1]);
          f[k] -= __half2float(k & 1 ? __high2half(h2) : __low2half(h2));
          if (!(f[k] == f[k])) f[k] = 0.0f;  // infinities and NaN are the first part's alone
        }
        p[x_rest / 16] =
            make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
      }
    });
  }
  if constexpr (PAIR != PAIR_NO) {
    if (tid < ZEROS / 16) reinterpret_cast<uint4*>(xs + (SILU ? 2 : 1) * x_rest)[tid] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();

  // ---- products -------------------------------------------------------------------------
  // The accumulator of the tensor core is off by more per addition than a rounded float32 sum; it
  // only runs over one step (128 columns), and the steps are added in float32.
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
  const uint8_t* xlane[NT];  // rows past the tokens read the last one: their columns are not stored
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int m = SILU == SILU_ROWS ? g >> 1 : 8 * n + g;
    xlane[n] = xs + (m < tokens ? m : tokens - 1) * pitch + gb * 256 + t * 16;
    if (SILU == SILU_ROWS && (g & 1)) xlane[n] += x_rest;
  }
  // One or two rows of x: the operand's eight columns are rows of x times lanes t, column 2 t + m holding
  // row m at lane t's places of K and 0 elsewhere. A sum then covers one lane's columns only, that is one
  // scale block per row in four instructions, and is multiplied by that block's scale: 12 float32
  // instructions per step instead of 32 f16 products, and weights go to the tensor core as they are decoded.
  // (2 x 4096 x 24576: 20.1 -> 19.2 us.)
  const uint8_t* const zeros = xs + (SILU ? 2 : 1) * x_rest;
  const bool holds = (g >> 1) == t;
  const uint8_t* const xpair = holds ? xs + (SILU ? (g & 1) * x_rest : (g & 1) < tokens ? (g & 1) * pitch : 0) + gb * 256 + t * 16
                                    : zeros + t * 16;
  const int xpair_step = holds ? 256 : 0;
  auto compute_pair = [&](int step, const uint8_t* codes, const uint8_t* scales) {
    float2 sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h2;
      const uint16_t two = *reinterpret_cast<const uint16_t*>(scales + 8 * i);
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
      sc[i] = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    }
    const uint4 q0 = *reinterpret_cast<const uint4*>(codes);
    const uint4 q1 = *reinterpret_cast<const uint4*>(codes + 8 * 128);
    const uint32_t c0[4] = {q0.x, q0.y, q0.z, q0.w};
    const uint32_t c1[4] = {q1.x, q1.y, q1.z, q1.w};
    const uint8_t* const xp = xpair + step * xpair_step;
    float sum[2][4];  // of the lane's two blocks
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {  // the two blocks in turn: neither waits for the other's sum
        const int w = 2 * b + h;
        uint32_t a0[4], a1[4];
        e2m1x8_to_f16x2(c0[w], a0);
        e2m1x8_to_f16x2(c1[w], a1);
        const uint4 xb = *reinterpret_cast<const uint4*>(xp + w * 64);
        if (h == 0) {
          mma_16x8x16_from0(sum[b], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
        } else {
          mma_16x8x16(sum[b], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
        }
        mma_16x8x16(sum[b], a0[2], a1[2], a0[3], a1[3], xb.z, xb.w);
      }
    }
    const float2 f = *reinterpret_cast<const float2*>(inv + (gb + step) * 8 * NT);  // of rows 0 and 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 s = sc[i >> 1];
      acc[0][i] = fmaf(fmaf(sum[1][i], s.y, sum[0][i] * s.x), i & 1 ? f.y : f.x, acc[0][i]);
    }
  };
  // Two rows with SiLU are four values per place of K, so the columns suffice for two halves of the lanes.
  // ldmatrix gives lanes t = 0, 1 and t = 2, 3 eight codes each of the same scale block: column 4 h + i holds part
  // i & 1 of row i / 2 at the places of lanes t / 2 = h, and a sum covers one block per row in two instructions.
  // (2 x 4096 x 24576: 16.7 us; with scales on the weights and eight columns of x 18.3, with twice the
  // instructions of compute_pair 19.5.)
  const bool in_half = (g >> 2) == (t >> 1);
  const int half_row = (g >> 1) & 1;
  const uint8_t* const xhalf =
      in_half ? xs + (half_row < tokens ? half_row : 0) * pitch + (g & 1) * x_rest + gb * 256 + t * 16 : zeros + t * 16;
  const int xhalf_step = in_half ? 256 : 0;
  const uint32_t half_scales = t & 2 ? 0x7531u : 0x6420u;
  auto compute_halves = [&](int step, uint32_t codes, const uint8_t* scales) {
    uint32_t c0[4], c1[4];
    ldmatrix_x4(codes, c0);
    ldmatrix_x4(codes + 8 * 128, c1);
    float2 sc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t four = __byte_perm(*reinterpret_cast<const uint32_t*>(scales + 8 * i),
                                        *reinterpret_cast<const uint32_t*>(scales + 64 + 8 * i), half_scales);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h2;
        const uint16_t two = static_cast<uint16_t>(four >> 16 * k);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
        sc[i][k] = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      }
    }
    const uint8_t* const xp = xhalf + step * xhalf_step;
    float sum[4][4];  // of the half's four blocks
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0[4], a1[4];
      e2m1x8_to_f16x2(c0[w], a0);
      e2m1x8_to_f16x2(c1[w], a1);
      const uint4 xb = *reinterpret_cast<const uint4*>(xp + w * 64);
      mma_16x8x16_from0(sum[w], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
      mma_16x8x16(sum[w], a0[2], a1[2], a0[3], a1[3], xb.z, xb.w);
    }
    const float f = inv[(gb + step) * 8 + (t & 1) * 2];  // of row t & 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 (&s)[2] = sc[i >> 1];
      const float one = fmaf(sum[3][i], s[1].y, fmaf(sum[2][i], s[1].x, fmaf(sum[1][i], s[0].y, sum[0][i] * s[0].x)));
      acc[0][i] = fmaf(one, f, acc[0][i]);
    }
  };
  auto compute = [&](int step, const uint8_t* codes, const uint8_t* scales) {
    uint32_t s2[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h2;
      const uint16_t two = *reinterpret_cast<const uint16_t*>(scales + 8 * i);
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
      s2[i][0] = __byte_perm(h2, h2, 0x1010);
      s2[i][1] = __byte_perm(h2, h2, 0x3232);
    }
    const uint4 q0 = *reinterpret_cast<const uint4*>(codes);
    const uint4 q1 = *reinterpret_cast<const uint4*>(codes + 8 * 128);
    const uint32_t c0[4] = {q0.x, q0.y, q0.z, q0.w};
    const uint32_t c1[4] = {q1.x, q1.y, q1.z, q1.w};
    float one[NT][4], rest[4];  // rest: with NT = 1 the second parts' sums do not wait for the first's
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0[4], a1[4];
      e2m1x8_to_f16x2(c0[w], a0);
      e2m1x8_to_f16x2(c1[w], a1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a0[j] = mul_f16x2(a0[j], s2[0][w >> 1]);
        a1[j] = mul_f16x2(a1[j], s2[1][w >> 1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 xb = *reinterpret_cast<const uint4*>(xlane[n] + step * 256 + w * 64);
        if (w == 0) {
          mma_16x8x16_from0(one[n], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
        } else {
          mma_16x8x16(one[n], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
        }
        mma_16x8x16(one[n], a0[2], a1[2], a0[3], a1[3], xb.z, xb.w);
        if constexpr (SILU == SILU_PARTS) {
          const uint4 xr = *reinterpret_cast<const uint4*>(xlane[n] + x_rest + step * 256 + w * 64);
          float (&to)[4] = NT == 1 ? rest : one[n];
          if (NT == 1 && w == 0) {
            mma_16x8x16_from0(to, a0[0], a1[0], a0[1], a1[1], xr.x, xr.y);
          } else {
            mma_16x8x16(to, a0[0], a1[0], a0[1], a1[1], xr.x, xr.y);
          }
          mma_16x8x16(to, a0[2], a1[2], a0[3], a1[3], xr.z, xr.w);
        }
      }
    }
    if constexpr (SILU == SILU_PARTS && NT == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) one[0][i] += rest[i];
    }
    const float* const factor = inv + (gb + step) * 8 * NT + 2 * t;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 f = *reinterpret_cast<const float2*>(factor + 8 * n);  // of rows 2 t and 2 t + 1
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(one[n][i], i & 1 ? f.y : f.x, acc[n][i]);
    }
  };
  // Value i of lane's fragment: weight row g or g + 8 of the strip, row 2 t or 2 t + 1 of x (PAIR: row 0 or 1);
  // with SILU_ROWS value 0 or 2, row t (PAIR: row 0)
  float bias[2] = {0.0f, 0.0f};
  auto load_bias = [&](int strip) {
    const int64_t row = static_cast<int64_t>(strip >> 3) * 128 + (g >> 2) * 32 + (strip & 7) * 4 + (g & 3);
    if (a.bias != nullptr) {
      if (row < a.N) bias[0] = __ldg(a.bias + row);
      if (row + 64 < a.N) bias[1] = __ldg(a.bias + row + 64);
    }
  };
  auto put = [&](int strip, int n, int i, float v) {
    if (SILU == SILU_ROWS && (i & 1)) return;
    // with PAIR the other lanes hold the same
    const int m = PAIR == PAIR_LANES   ? 8 * t * 2 + (SILU == SILU_ROWS ? 0 : i & 1)
                  : SILU == SILU_ROWS  ? t  // PAIR_HALVES has two rows, lanes 2 and 3 none
                                       : 8 * n + 2 * t + (i & 1);
    const int64_t row = static_cast<int64_t>(strip >> 3) * 128 + (g >> 2) * 32 + (i >> 1) * 64 + (strip & 7) * 4 + (g & 3);
    if (m >= tokens || row >= a.N) return;
    v += bias[i >> 1];
    const int64_t at = (m0 + m) * a.ldd + row;
    if (a.out_kind == 2) {
      static_cast<float*>(a.D)[at] = v;
    } else if (a.out_kind == 1) {
      static_cast<__half*>(a.D)[at] = __float2half_rn(v);
    } else {
      static_cast<__nv_bfloat16*>(a.D)[at] = __float2bfloat16_rn(v);
    }
  };

  if (cluster > 1) cluster_wait();  // every CTA has started: its shared memory can be written to
  int buf = 0, round_buf = 0, in_round = 0;
  int it = 0, round_base = 0;  // strip iteration, first iteration of the round
  // The end of a strip: its pieces of K are joined over the warps, and over the cluster.
  auto finish = [&]() {
    const int strip = it * a.strips_at_once + cid * rows_at_once + wr;
    const bool have = strip < a.strips;
    float sum[4 * NT];
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) {
      sum[i] = acc[i >> 2][i & 3];
      acc[i >> 2][i & 3] = 0.0f;
    }
    if constexpr (SILU == SILU_ROWS) {  // the two parts of a row
      sum[0] += sum[1];
      sum[2] += sum[3];
      sum[1] = sum[3] = 0.0f;
    }
    bool mine = have;
    if (kwarps > 1) {
      float* slot = red + ((buf * WARPS + warp) * 32 + lane) * 4 * NT;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        *reinterpret_cast<float4*>(slot + 4 * i) = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
      named_barrier(1 + wr, 32 * kwarps);
      // the warps of a strip take turns at adding up its pieces
      mine = have && wk == (it & (kwarps - 1));
      if (mine) {
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) sum[i] = 0.0f;
        for (int w = 0; w < kwarps; ++w) {
          const float* p = red + ((buf * WARPS + wr * kwarps + w) * 32 + lane) * 4 * NT;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(p + 4 * i);
            sum[4 * i] += f.x;
            sum[4 * i + 1] += f.y;
            sum[4 * i + 2] += f.z;
            sum[4 * i + 3] += f.w;
          }
        }
      }
      buf ^= 1;
    }
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) {
        // the lanes' or halves' blocks
        if constexpr (PAIR == PAIR_LANES) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        if constexpr (PAIR != PAIR_NO) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        sum[i] *= G;
      }
      if (cluster == 1) {
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) put(strip, i >> 2, i & 3, sum[i]);
      } else {
        // strip s of the round is added up by CTA s modulo `cluster`: its piece goes there
        const int s = in_round + wr, at = (s & ~(cluster - 1)) + rank;
        const uint32_t there =
            mapa_shared(smem_u32(part + ((round_buf * ROUND + at) * 32 + lane) * 4 * NT), s & (cluster - 1));
#pragma unroll
        for (int i = 0; i < NT; ++i)
          st_cluster_f32x4(there + 16 * i, sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
      }
    }
    if (cluster > 1) {
      in_round += rows_at_once;
      if (in_round + rows_at_once > ROUND || it == a.iters - 1) {
        // Every CTA's pieces of this round's strips are written. The round after the next uses their places
        // again, behind the next round's barrier, which no CTA reaches before it has read them.
        cluster_sync_all();
        for (int s = rank + cluster * warp; s < in_round; s += cluster * WARPS) {
          const int st = (round_base + s / rows_at_once) * a.strips_at_once + cid * rows_at_once + s % rows_at_once;
          if (st >= a.strips) continue;
          load_bias(st);
          const float* p = part + ((round_buf * ROUND + (s & ~(cluster - 1))) * 32 + lane) * 4 * NT;
          float all[4 * NT];
#pragma unroll
          for (int i = 0; i < 4 * NT; ++i) all[i] = 0.0f;
          for (int c = 0; c < cluster; ++c, p += 128 * NT) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const float4 f = *reinterpret_cast<const float4*>(p + 4 * i);
              all[4 * i] += f.x;
              all[4 * i + 1] += f.y;
              all[4 * i + 2] += f.z;
              all[4 * i + 3] += f.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 4 * NT; ++i) put(st, i >> 2, i & 3, all[i]);
        }
        round_buf ^= 1;
        in_round = 0;
        round_base = it + 1;
      }
    }
    ++it;
  };

  // the lane's places in a chunk: its columns of weight row g (row g + 8 is 1024 bytes further), its scales
  const uint8_t* const my_codes = ring + warp * (BUFFERS * CHUNK) + g * 128 + (g & 1) * 64 + t * 16;
  const int other = (g & 1) ? -64 : 64;  // to the chunk's second step
  const uint8_t* const my_scales = ring + warp * (BUFFERS * CHUNK) + CODES + (g & 3) * 16 + (g >> 2) * 4 +
                                   (PAIR == PAIR_HALVES ? 0 : (t >> 1) * 64 + (t & 1) * 2);
  // PAIR_HALVES: the row that this lane names for ldmatrix, 16 bytes of row lane & 7
  const uint32_t my_halves = my_ring, half_at = (lane & 7) * 128 + ((lane >> 3) ^ (lane & 7)) * 16;
  int slot = 0;
  while (it < a.iters) {
    const int strip = it * a.strips_at_once + cid * rows_at_once + wr;
    if (cluster == 1 && wk == (it & (kwarps - 1)) && strip < a.strips) load_bias(strip);
    for (int c = 0; c < chunks; ++c) {
      copy_async_wait<BUFFERS - 1>();
      __syncwarp();  // other lanes copied what this one reads
      const uint8_t* const codes = my_codes + slot * CHUNK;
      const uint8_t* const scales = my_scales + slot * CHUNK;
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const int step = c * STEPS + j;
        if (step < my_groups) {
          if constexpr (PAIR == PAIR_HALVES) {
            compute_halves(step, my_halves + slot * CHUNK + (j ? half_at ^ 64 : half_at), scales + j * 128);
          } else if constexpr (PAIR == PAIR_LANES) {
            compute_pair(step, codes + j * other, scales + j * 128);
          } else {
            compute(step, codes + j * other, scales + j * 128);
          }
        }
      }
      __syncwarp();  // every lane has read the chunk
      load(slot);
      slot = (slot + 1) & (BUFFERS - 1);
    }
    finish();
  }
}

}  // namespace nvfp4
