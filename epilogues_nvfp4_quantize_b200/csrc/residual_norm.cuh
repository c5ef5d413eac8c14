// residual_norm: the residual stream between two blocks of a layer, and its gradient.
//
//   x' = alpha x + gate[b] y~        y~ = y, or y rsqrt(mean y^2 + eps) w_post
//   h  = n(x') w (1 + scale[b]) + shift[b],   n = LayerNorm or RMSNorm over the row
//
// b is the row's sequence (a modulation vector each). x' is rounded to the stream's type once,
// and the norm reads the rounded value: the gradient, which only has the stored x', then
// differentiates exactly what was computed. h is rounded to bf16 once; its NVFP4 form quantises
// those bf16 values, as every re-quantised output of this library does.
// Sums, means and reciprocal roots are float32; the variance is taken from centred values (a
// second pass over registers), so a mean much larger than the spread costs no digits.
#pragma once

#include "ptx.cuh"
#include "codec.cuh"
#include "quantize.cuh"

namespace nvfp4 {

struct NormArgs {
  int64_t rows, cols;
  int64_t batches;        // sequences
  int64_t rows_per_batch; // of each sequence, when offsets is null
  const int* offsets;     // batches + 1 row offsets, or null
  const void* x;          // the stream (bf16 or float32)
  int64_t ldx;
  const uint16_t* y;      // the branch (bf16), or null
  int64_t ldy;
  const void* gate;       // batches x cols (bf16 or float32, see mod_f32), or null (1)
  const void* scale;      // or null (0)
  const void* shift;      // or null (0)
  int64_t ldgate, ldscale, ldshift;
  int mod_f32;
  int post;               // RMSNorm on the branch
  const float* w_post;    // or null (1)
  const float* w;         // or null (1)
  int norm;               // 0 none, 1 LayerNorm, 2 RMSNorm
  float alpha, eps;
  void* x_out;            // or null
  int64_t ldxo;
  uint16_t* h;            // or null
  int64_t ldh;
  uint8_t* q_codes;       // NVFP4 output, or null
  uint8_t* q_sf;
  const float* q_gscale;
  float* stats;           // rows x 4: mean, rstd, rstd of the branch, 0; or null
};

enum NormKind { NORM_NONE = 0, NORM_LAYER = 1, NORM_RMS = 2 };

// Sequence of a row, or -1 when it has none (rows before the first offset or behind the last). All
// lanes of a warp ask for the same row: each step probes 32 offsets at once, so up to 31 sequences
// take one load. The offsets come from the device and are not checked: whatever they hold, the
// answer is -1 or in [0, batches).
__device__ __forceinline__ int64_t norm_sequence(const int* offsets, int64_t batches, int64_t rows_per_batch,
                                                 int64_t row) {
  if (offsets == nullptr) {  // rows fit in 31 bits
    return static_cast<uint32_t>(row) / static_cast<uint32_t>(rows_per_batch);
  }
  int64_t lo = 0, hi = batches + 1;  // the number of offsets <= row is in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) >> 5, at = lo + (threadIdx.x & 31) * step;
    const int c = __popc(__ballot_sync(0xffffffffu, at < hi && static_cast<int64_t>(__ldg(offsets + at)) <= row));
    if (c == 0) {
      hi = lo;
    } else {
      const int64_t end = lo + c * step;
      lo += (c - 1) * step + 1;
      hi = end < hi ? end : hi;
    }
  }
  return lo > batches ? -1 : lo - 1;
}

// Eight values of the stream.
template <class ST>
struct Stream8;
template <>
struct Stream8<uint16_t> {
  uint4 q;
  __device__ void load(const void* base, int64_t at) {
    q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
  }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  // Rounds v to the stream's type (in place) and holds the result.
  __device__ void round(float (&v)[8]) {
    q = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
    get(v);
  }
  __device__ void store(void* base, int64_t at) const {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = q;
  }
};
template <>
struct Stream8<float> {
  float4 q[2];
  __device__ void load(const void* base, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    q[0] = p[0];
    q[1] = p[1];
  }
  __device__ void get(float (&v)[8]) const {
    v[0] = q[0].x, v[1] = q[0].y, v[2] = q[0].z, v[3] = q[0].w;
    v[4] = q[1].x, v[5] = q[1].y, v[6] = q[1].z, v[7] = q[1].w;
  }
  __device__ void round(float (&v)[8]) {
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ void store(void* base, int64_t at) const {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = q[0];
    p[1] = q[1];
  }
};

__device__ __forceinline__ void load8_bf16(const uint16_t* p, float (&v)[8]) {
  Stream8<uint16_t> s;
  s.load(p, 0);
  s.get(v);
}

// Eight modulation values at column c of sequence b.
__device__ __forceinline__ void load8_mod(const void* base, int mod_f32, int64_t at, float (&v)[8]) {
  if (mod_f32) {
    Stream8<float> s;
    s.load(base, at);
    s.get(v);
  } else {
    Stream8<uint16_t> s;
    s.load(base, at);
    s.get(v);
  }
}
__device__ __forceinline__ void load8_f32(const float* p, float (&v)[8]) {
  Stream8<float> s;
  s.load(p, 0);
  s.get(v);
}

__device__ __forceinline__ void store8_f32(float* p, float (&v)[8]) {
  Stream8<float> s;
  s.round(v);
  s.store(p, 0);
}

// Sum over the threads of a row: one warp (ONE_WARP), or all of the CTA's (red: 32 floats,
// flipped between two halves by the caller so that one barrier per sum suffices).
template <bool ONE_WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (ONE_WARP) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One row per CTA (ONE_WARP: per warp); thread t holds the eight columns at 8 t, and with NV > 1
// those at 8 (t + i threads).
template <class ST, int NV, bool ONE_WARP>
__global__ void __launch_bounds__(ONE_WARP ? 128 : 1024) residual_norm_kernel(const NormArgs a) {
  __shared__ float red[3][32];
  griddep_launch_dependents();
  griddep_wait();
  const int threads = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = ONE_WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                               : static_cast<int64_t>(blockIdx.x);
  const int64_t nkb = a.cols >> 4;
  if (row >= a.rows) {  // rows that pad the block scales to 128 (their scales are 0)
    if (a.q_codes != nullptr && row < ((a.rows + 127) & ~int64_t(127))) {
      for (int64_t g = t; g < (a.cols >> 6); g += threads)
        *reinterpret_cast<uint32_t*>(a.q_sf + sf_word_offset(row, 4 * g, nkb)) = 0u;
    }
    return;
  }
  const int64_t b = norm_sequence(a.offsets, a.batches, a.rows_per_batch, row);
  if (b < 0) return;

  Stream8<ST> xs[NV];
  float v[NV][8];
  uint4 yq[NV];
  bool live[NV];
  int64_t col[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = 8 * static_cast<int64_t>(t + i * threads);
    live[i] = col[i] < a.cols;
    if (live[i]) {
      xs[i].load(a.x, row * a.ldx + col[i]);
      if (a.y != nullptr) yq[i] = *reinterpret_cast<const uint4*>(a.y + row * a.ldy + col[i]);
    }
  }
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  float rstd_y = 1.0f;
  if (a.y != nullptr) {
    if (a.post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live[i]) continue;
        const uint32_t w[4] = {yq[i].x, yq[i].y, yq[i].z, yq[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fmaf(bf16_lo(w[k]), bf16_lo(w[k]), fmaf(bf16_hi(w[k]), bf16_hi(w[k]), ss));
      }
      rstd_y = rsqrtf(row_sum<ONE_WARP>(ss, red[0]) * inv_n + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      float g[8], yv[8];
      Stream8<uint16_t> ys;
      ys.q = yq[i];
      ys.get(yv);
      xs[i].get(v[i]);
      if (a.post) {
#pragma unroll
        for (int k = 0; k < 8; ++k) yv[k] *= rstd_y;
        if (a.w_post != nullptr) {
          load8_f32(a.w_post + col[i], g);
#pragma unroll
          for (int k = 0; k < 8; ++k) yv[k] *= g[k];
        }
      }
      if (a.gate != nullptr) {
        load8_mod(a.gate, a.mod_f32, b * a.ldgate + col[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) yv[k] *= g[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = fmaf(a.alpha, v[i][k], yv[k]);
      xs[i].round(v[i]);
      if (a.x_out != nullptr) xs[i].store(a.x_out, row * a.ldxo + col[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      xs[i].get(v[i]);
      if (a.x_out != nullptr) xs[i].store(a.x_out, row * a.ldxo + col[i]);
    }
  }
  float mean = 0.0f, rstd = 1.0f;
  if (a.norm != NORM_NONE) {
    if (a.norm == NORM_LAYER) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live[i]) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[i][k];
      }
      mean = row_sum<ONE_WARP>(s, red[1]) * inv_n;
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] -= mean;
        ss = fmaf(v[i][k], v[i][k], ss);
      }
    }
    rstd = rsqrtf(row_sum<ONE_WARP>(ss, red[2]) * inv_n + a.eps);
  }
  if (a.stats != nullptr && t == 0) *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(mean, rstd, rstd_y, 0.0f);
  if (a.norm == NORM_NONE) return;

  float G = 0.0f, enc = 0.0f;
  if (a.q_codes != nullptr) {
    G = *a.q_gscale;
    enc = scale_encode_factor(G);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Stream8<uint16_t> out;
    out.q = make_uint4(0u, 0u, 0u, 0u);
    if (live[i]) {
      float g[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] *= rstd;
      if (a.w != nullptr) {
        load8_f32(a.w + col[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] *= g[k];
      }
      if (a.scale != nullptr) {
        load8_mod(a.scale, a.mod_f32, b * a.ldscale + col[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = fmaf(v[i][k], g[k], v[i][k]);
      }
      if (a.shift != nullptr) {
        load8_mod(a.shift, a.mod_f32, b * a.ldshift + col[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] += g[k];
      }
      out.round(v[i]);
      if (a.h != nullptr) out.store(a.h, row * a.ldh + col[i]);
    }
    if (a.q_codes != nullptr) {
      // a block of 16 is two lanes, a scale word (64 columns) eight: cols % 64 == 0, so each
      // group of eight lanes is live as a whole
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, live[i] ? fabsf(v[i][k]) : 0.0f);
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const uint32_t s = block_scale_code(amax, enc);
      const float r = block_inv_scale(s, G);
      const int lane = threadIdx.x & 31;
      uint32_t word = (lane & 1) ? 0u : s << (4 * (lane & 7));
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      if (live[i]) {
        const uint32_t codes = r > 0.0f ? block_codes8(v[i], r) : 0u;
        *reinterpret_cast<uint32_t*>(a.q_codes + row * (a.cols >> 1) + (col[i] >> 1)) = codes;
        if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(a.q_sf + sf_word_offset(row, col[i] >> 4, nkb)) = word;
      }
    }
  }
}

// =====================================================================================
// Gradient. With xhat = (x' - mean) rstd, d = dh w (1 + scale), yh the normalised branch (or y):
//   T       = dx' + rstd (d - mean(d) [LayerNorm] - xhat mean(d xhat))     gradient of x'
//   dx      = alpha T
//   dy      = gate T, or with the branch's norm rstd_y (a - yh mean(a yh)), a = gate w_post T
//   dshift  = sum_b dh,  dscale = sum_b dh xhat w,  dgate = sum_b T yh w_post
//   dw      = sum dh xhat (1 + scale),  dw_post = sum gate T yh
// so three sums over a sequence's rows (dh, dh xhat, T yh) give every parameter's gradient.
// mean(a yh) depends on T; it is expanded into sums that do not (six row sums in all), so that a
// row needs one reduction only.
//
// Rows are cut into `chunks` contiguous pieces, one CTA each; a thread keeps its columns and
// adds up the three sums in registers over the rows of its piece. Where a sequence ends, the sums
// go to slot chunk + sequence of the workspace (that index grows with every piece, so no two
// pieces share one); norm_grad_reduce_kernel adds a sequence's slots in their order. No atomics:
// the same inputs give the same bits.
// =====================================================================================
struct NormGradArgs {
  int64_t rows, cols, batches, rows_per_batch;
  const int* offsets;
  const void* x;          // x', the stored stream
  int64_t ldx;
  const void* dxo;        // gradient of x' from what follows (the stream's type), or null (0)
  int64_t lddxo;
  const uint16_t* dh;     // or null: no norm
  int64_t lddh;
  const uint16_t* y;      // or null: no branch
  int64_t ldy;
  const void* gate;
  const void* scale;
  int64_t ldgate, ldscale;
  int mod_f32;
  int post;
  const float* w_post;
  const float* w;
  int norm;
  float alpha;
  const float* stats;
  void* dx;
  int64_t lddx;
  uint16_t* dy;
  int64_t lddy;
  float* dgate;           // batches x cols, or null; likewise below
  float* dscale;
  float* dshift;
  int64_t lddgate, lddscale, lddshift;
  float* dw;              // cols, or null
  float* dw_post;
  int chunks;
  int stages;             // row buffers of the ring
  float* seq_part;        // (chunks + batches) x 3 x cols, or null (no sums)
  float* w_part;          // chunks x 2 x cols, or null (neither dw nor dw_post)
};

__device__ __forceinline__ int64_t norm_chunk_row(int64_t rows, int chunks, int64_t g) { return rows * g / chunks; }

namespace normcfg {
constexpr int GRAD_THREADS = 512;        // threads per SM that the gradient kernel's registers allow
constexpr int GRAD_MAX_STAGES = 8;
constexpr int REDUCE_ROWS = 32;
constexpr int GRAD_SMEM = 220 * 1024;    // per SM, for its CTAs' row buffers and GRAD_OTHER each
constexpr int GRAD_OTHER = 3584;         // a CTA's static and reserved shared memory
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
}  // namespace normcfg

// Bytes of one row's buffer: the stream, its gradient, the gradient of h, the branch, the statistics
// (absent ones take no room).
__host__ __device__ constexpr int64_t norm_grad_stage(int64_t cols, int elem, bool dxo, bool dh, bool y) {
  return cols * (elem * (dxo + dh) + 2 * (dh + y)) + 16;
}

// Sums over the CTA of the first N of six values per thread (N = 2 or 6); every thread gets them.
// Within a warp, each of the first log2 exchanges halves the values a lane keeps (9 shuffles for
// six sums instead of 30); lane 4 k then holds sum k. `red` holds 32 x 8 floats.
template <int N>
__device__ __forceinline__ void cta_sums(float (&s)[6], float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float v;
  if constexpr (N == 6) {
    float a4[4], a2[2];
    const bool h16 = (lane & 16) != 0, h8 = (lane & 8) != 0, h4 = (lane & 4) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = s[k], hi = k < 2 ? s[k + 4] : 0.0f;
      a4[k] = (h16 ? hi : lo) + __shfl_xor_sync(0xffffffffu, h16 ? lo : hi, 16);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      a2[k] = (h8 ? a4[k + 2] : a4[k]) + __shfl_xor_sync(0xffffffffu, h8 ? a4[k] : a4[k + 2], 8);
    v = (h4 ? a2[1] : a2[0]) + __shfl_xor_sync(0xffffffffu, h4 ? a2[0] : a2[1], 4);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    if ((lane & 3) == 0) red[warp * 8 + (lane >> 2)] = v;
  } else {
    const bool h16 = (lane & 16) != 0;
    v = (h16 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, h16 ? s[0] : s[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((lane & 15) == 0) red[warp * 8 + (lane >> 4)] = v;
  }
  __syncthreads();
  v = 0.0f;
  for (int w = lane >> 3; w < warps; w += 4) v += red[w * 8 + (lane & 7)];
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = __shfl_sync(0xffffffffu, v, k);
}

// A CTA walks the rows of its piece; thread t holds the eight columns at 8 t (and with NV > 1 those
// at 8 (t + i threads)). Rows come through a ring of row buffers, filled by bulk copies (one per
// tensor and row, issued by one thread `stages` rows ahead), so the loads of the coming rows are in
// flight while a row is reduced. The one barrier of a row's reduction is also what frees its buffer:
// every thread has read its values by then.
// POST: the branch has its norm (six row sums, else two). With NV = 1 the sequence's constants per
// column stay in registers, else they are read again for each row (from L1).
template <class ST, int NV, bool POST>
__global__ void __launch_bounds__(normcfg::GRAD_THREADS) residual_norm_grad_kernel(const NormGradArgs a) {
  using namespace normcfg;
  extern __shared__ __align__(128) uint8_t norm_rows[];
  __shared__ float red[2][32 * 8];
  __shared__ __align__(8) uint64_t full[GRAD_MAX_STAGES];
  __shared__ int abort_flag;
  griddep_launch_dependents();
  griddep_wait();
  const int g = blockIdx.x;
  const int64_t r0 = norm_chunk_row(a.rows, a.chunks, g), r1 = norm_chunk_row(a.rows, a.chunks, g + 1);
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  const bool has_dxo = a.dxo != nullptr, has_dh = a.dh != nullptr, has_y = a.y != nullptr;
  // the parts of a row buffer
  const uint32_t stream_bytes = static_cast<uint32_t>(a.cols * sizeof(ST)), half_bytes = static_cast<uint32_t>(a.cols * 2);
  const uint32_t at_dxo = has_dh ? stream_bytes : 0u, at_dh = at_dxo + (has_dxo ? stream_bytes : 0u);
  const uint32_t at_y = at_dh + (has_dh ? half_bytes : 0u), at_stats = at_y + (has_y ? half_bytes : 0u);
  const uint32_t stage_bytes = at_stats + 16u;

  auto fetch = [&](int64_t row, int stage) {  // one thread
    uint8_t* to = norm_rows + stage * stage_bytes;
    uint64_t* bar = &full[stage];
    mbar_arrive_expect_tx(bar, stage_bytes);
    if (has_dh) {
      bulk_load(to, static_cast<const ST*>(a.x) + row * a.ldx, stream_bytes, bar);
      bulk_load(to + at_dh, a.dh + row * a.lddh, half_bytes, bar);
    }
    if (has_dxo) bulk_load(to + at_dxo, static_cast<const ST*>(a.dxo) + row * a.lddxo, stream_bytes, bar);
    if (has_y) bulk_load(to + at_y, a.y + row * a.ldy, half_bytes, bar);
    bulk_load(to + at_stats, a.stats + 4 * row, 16u, bar);
  };
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
    for (int i = 0; i < a.stages && r0 + i < r1; ++i) fetch(r0 + i, i);
  }
  __syncthreads();

  bool live[NV];
  int col[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = 8 * static_cast<int>(threadIdx.x + i * blockDim.x);
    live[i] = col[i] < a.cols;
  }
  float s_dh[NV][8], s_dhx[NV][8], s_ty[NV][8];  // sums over the current sequence's rows
  constexpr int NC = NV == 1 ? 1 : 0;
  float c_w[NC + 1][8], c_g[NC + 1][8], c_a[NC + 1][8];  // w (1 + scale), the gate, gate w_post
  bool first_flush = true;
  int64_t b = -1, seq_end = r0;

  // the sequence's constants of vector i
  auto constants = [&](int i, float (&cw)[8], float (&gt)[8], float (&ag)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) cw[k] = gt[k] = 1.0f;
    if (a.scale != nullptr) {
      load8_mod(a.scale, a.mod_f32, b * a.ldscale + col[i], cw);
#pragma unroll
      for (int k = 0; k < 8; ++k) cw[k] += 1.0f;
    }
    if (a.w != nullptr) {
      load8_f32(a.w + col[i], ag);
#pragma unroll
      for (int k = 0; k < 8; ++k) cw[k] *= ag[k];
    }
    if (a.gate != nullptr) load8_mod(a.gate, a.mod_f32, b * a.ldgate + col[i], gt);
    if constexpr (POST) {
#pragma unroll
      for (int k = 0; k < 8; ++k) ag[k] = 1.0f;
      if (a.w_post != nullptr) load8_f32(a.w_post + col[i], ag);
#pragma unroll
      for (int k = 0; k < 8; ++k) ag[k] *= gt[k];
    }
  };
  auto flush = [&]() {
    if (a.seq_part == nullptr) return;  // no sums are asked for
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      float* p = a.seq_part + (g + b) * 3 * a.cols + col[i];
      store8_f32(p, s_dh[i]);
      store8_f32(p + a.cols, s_dhx[i]);
      store8_f32(p + 2 * a.cols, s_ty[i]);
      if (a.w_part != nullptr) {
        float* q = a.w_part + static_cast<int64_t>(g) * 2 * a.cols + col[i];
        float w0[8], p0[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w0[k] = 0.0f, p0[k] = 1.0f;
        if (a.scale != nullptr) load8_mod(a.scale, a.mod_f32, b * a.ldscale + col[i], w0);
        if (a.gate != nullptr) load8_mod(a.gate, a.mod_f32, b * a.ldgate + col[i], p0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          w0[k] = (1.0f + w0[k]) * s_dhx[i][k];
          p0[k] *= s_ty[i][k];
        }
        if (!first_flush) {
          float o[8];
          load8_f32(q, o);
#pragma unroll
          for (int k = 0; k < 8; ++k) w0[k] += o[k];
          load8_f32(q + a.cols, o);
#pragma unroll
          for (int k = 0; k < 8; ++k) p0[k] += o[k];
        }
        store8_f32(q, w0);
        store8_f32(q + a.cols, p0);
      }
    }
    first_flush = false;
  };

  int stage = 0;
  uint32_t phase = 0u;
  for (int64_t row = r0; row < r1; ++row) {
    bool skip = false;
    if (row >= seq_end) {
      if (b >= 0) flush();
      b = norm_sequence(a.offsets, a.batches, a.rows_per_batch, row);
      if (b < 0) {  // rows without a sequence are left as they are
        seq_end = row + 1;
        skip = true;
      } else {
        seq_end = a.offsets == nullptr ? (b + 1) * a.rows_per_batch : static_cast<int64_t>(a.offsets[b + 1]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int k = 0; k < 8; ++k) s_dh[i][k] = s_dhx[i][k] = s_ty[i][k] = 0.0f;
          if constexpr (NV == 1) {
            if (live[0]) constants(0, c_w[0], c_g[0], c_a[0]);
          }
        }
      }
    }
    (void)mbar_wait(&full[stage], phase, &abort_flag, WAIT_LIMIT_NS, 80);
    const uint8_t* buf = norm_rows + stage * stage_bytes;
    if (skip) {
      __syncthreads();
    } else {
      const float4 st = *reinterpret_cast<const float4*>(buf + at_stats);
      const float mean = st.x, rstd = st.y, rstd_y = POST ? st.z : 1.0f;
      float xh[NV][8], d[NV][8], t[NV][8], yh[NV][8];
      float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) xh[i][k] = d[i][k] = t[i][k] = yh[i][k] = 0.0f;
        if (!live[i]) continue;
        if constexpr (NV > 1) constants(i, c_w[0], c_g[0], c_a[0]);
        Stream8<ST> v;
        if (has_dxo) {
          v.load(buf + at_dxo, col[i]);
          v.get(t[i]);
        }
        if (has_y) {
          load8_bf16(reinterpret_cast<const uint16_t*>(buf + at_y) + col[i], yh[i]);
          if constexpr (POST) {
#pragma unroll
            for (int k = 0; k < 8; ++k) yh[i][k] *= rstd_y;
          }
        }
        if (has_dh) {
          v.load(buf, col[i]);
          v.get(xh[i]);
          load8_bf16(reinterpret_cast<const uint16_t*>(buf + at_dh) + col[i], d[i]);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            xh[i][k] = (xh[i][k] - mean) * rstd;
            s_dh[i][k] += d[i][k];
            s_dhx[i][k] = fmaf(d[i][k], xh[i][k], s_dhx[i][k]);
            d[i][k] *= c_w[0][k];
            s[0] += d[i][k];
            s[1] = fmaf(d[i][k], xh[i][k], s[1]);
          }
        }
        if constexpr (POST) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float ay = c_a[0][k] * yh[i][k];
            s[2] = fmaf(ay, t[i][k], s[2]);
            s[3] = fmaf(ay, d[i][k], s[3]);
            s[4] += ay;
            s[5] = fmaf(ay, xh[i][k], s[5]);
          }
        }
      }
      cta_sums<POST ? 6 : 2>(s, red[static_cast<int>(row - r0) & 1]);
      const float m1 = a.norm == NORM_LAYER ? s[0] * inv_n : 0.0f, m2 = s[1] * inv_n;
      const float m3 = POST ? (s[2] + rstd * (s[3] - m1 * s[4] - m2 * s[5])) * inv_n : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live[i]) continue;
        if constexpr (NV > 1) constants(i, c_w[0], c_g[0], c_a[0]);
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (has_dh) t[i][k] = fmaf(rstd, d[i][k] - m1 - xh[i][k] * m2, t[i][k]);
          s_ty[i][k] = fmaf(t[i][k], yh[i][k], s_ty[i][k]);
          o[k] = a.alpha * t[i][k];
        }
        if (a.dx != nullptr) {
          Stream8<ST> v;
          v.round(o);
          v.store(a.dx, row * a.lddx + col[i]);
        }
        if (a.dy != nullptr) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = POST ? rstd_y * (c_a[0][k] * t[i][k] - yh[i][k] * m3) : c_g[0][k] * t[i][k];
          Stream8<uint16_t> v;
          v.round(o);
          v.store(a.dy, row * a.lddy + col[i]);
        }
      }
    }
    // every thread has passed this row's barrier, so its buffer takes the next row
    if (threadIdx.x == 0 && row + a.stages < r1) fetch(row + a.stages, stage);
    if (++stage == a.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (b >= 0) flush();
  if (a.w_part != nullptr && first_flush) {  // none of this piece's rows has a sequence
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      for (int k = 0; k < 8; ++k) {
        a.w_part[static_cast<int64_t>(g) * 2 * a.cols + col[i] + k] = 0.0f;
        a.w_part[(static_cast<int64_t>(g) * 2 + 1) * a.cols + col[i] + k] = 0.0f;
      }
    }
  }
}

// Adds up the slots of each sequence and the pieces' weight sums. Block (x, y): columns 32 x and
// on; y < gridDim.y - 1 takes the sequences y, y + gridDim.y - 1, ..., the last y the weights.
// 32 warps share the slots, one column per lane, and are joined in a fixed order (warp c then adds
// column c over the warps). With 148 to 2368 slots it is the latency of a thread's loads one after
// another that counts: 8 warps with 4 loads in flight took 12 us for 296 slots of 2048 columns.
__global__ void __launch_bounds__(32 * normcfg::REDUCE_ROWS) norm_grad_reduce_kernel(const NormGradArgs a) {
  using normcfg::REDUCE_ROWS;
  __shared__ float red[3][REDUCE_ROWS][33];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;        // while adding slots
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + warp;        // while joining
  const bool live = col < a.cols, last = lane == 0 && out < a.cols;
  auto total = [&](int k) {
    float v = red[k][lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  if (blockIdx.y == gridDim.y - 1) {
    float s0 = 0.0f, s1 = 0.0f;
    if (live && a.w_part != nullptr) {
      const float* p = a.w_part + static_cast<int64_t>(warp) * 2 * a.cols + col;
#pragma unroll 10
      for (int g = warp; g < a.chunks; g += REDUCE_ROWS, p += 2 * REDUCE_ROWS * a.cols) {
        s0 += p[0];
        s1 += p[a.cols];
      }
    }
    red[0][warp][lane] = s0;
    red[1][warp][lane] = s1;
    __syncthreads();
    s0 = total(0);
    s1 = total(1);
    if (last && a.dw != nullptr) a.dw[out] = s0;
    if (last && a.dw_post != nullptr) a.dw_post[out] = s1;
    return;
  }
  for (int64_t b = blockIdx.y; b < a.batches; b += gridDim.y - 1) {
    int64_t s = a.offsets == nullptr ? b * a.rows_per_batch : static_cast<int64_t>(a.offsets[b]);
    int64_t e = a.offsets == nullptr ? s + a.rows_per_batch : static_cast<int64_t>(a.offsets[b + 1]);
    if (s < 0) s = 0;
    if (e > a.rows) e = a.rows;
    float v[3] = {0.0f, 0.0f, 0.0f};
    if (s < e) {
      // pieces that hold rows of [s, e) (every piece has rows): from estimates
      int g0 = static_cast<int>(s * a.chunks / a.rows), g1 = static_cast<int>((e - 1) * a.chunks / a.rows);
      while (norm_chunk_row(a.rows, a.chunks, g0 + 1) <= s) ++g0;
      while (g1 + 1 < a.chunks && norm_chunk_row(a.rows, a.chunks, g1 + 1) < e) ++g1;
      if (live) {
        const float* p = a.seq_part + (g0 + warp + b) * 3 * a.cols + col;
#pragma unroll 5
        for (int g = g0 + warp; g <= g1; g += REDUCE_ROWS, p += 3 * REDUCE_ROWS * a.cols) {
          v[0] += p[0];
          v[1] += p[a.cols];
          v[2] += p[2 * a.cols];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) red[k][warp][lane] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = total(k);
    if (last) {
      if (a.dshift != nullptr) a.dshift[b * a.lddshift + out] = v[0];
      if (a.dscale != nullptr) a.dscale[b * a.lddscale + out] = v[1] * (a.w != nullptr ? a.w[out] : 1.0f);
      if (a.dgate != nullptr)
        a.dgate[b * a.lddgate + out] = v[2] * (a.post && a.w_post != nullptr ? a.w_post[out] : 1.0f);
    }
    __syncthreads();
  }
}

}  // namespace nvfp4
