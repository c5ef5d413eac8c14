// residual_norm: the residual stream between two blocks of a layer, and its gradient.
//
//   x' = alpha x + gate[b] y~        y~ = y, or y rsqrt(mean y^2 + eps) w_post
//   h  = n(x') w (1 + scale[b]) + shift[b],   n = LayerNorm or RMSNorm over the row
//
// b is the row's sequence (a modulation vector each). x' is rounded to the stream's type once,
// and the norm reads the rounded value: the gradient, which only has the stored x', then
// differentiates exactly what was computed. h is rounded to bf16 once; its NVFP4 form quantises
// those bf16 values, as every re-quantised output of this library does.
// Sums, means and reciprocal roots are float32; the variance is taken from centred values (about the
// row's mean, or about each warp's and joined), so a mean much larger than the spread costs no digits.
//
// All of it is HBM-bound: forward 2 + 2 + 2 + 2 bytes per value in bf16 (x, y, x', h), gradient 12
// (x', y, dx', dh, dx, dy).
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
  int chunks, stages;     // ring kernel: pieces of the rows, row buffers
  int64_t chunk_rows;     // rows of a piece, and how many pieces have one more
  int chunk_extra;
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

// Sum over the threads of a row: one warp (ONE_WARP), or all of the CTA's (red: 32 floats that no other
// sum uses, so that one barrier suffices).
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

// NVFP4 codes and scale of the eight bf16 values v at column col of a row. A block of 16 is two
// lanes, a scale word (64 columns) eight: cols % 64 == 0, so each group of eight lanes is live as a
// whole. All lanes of the warp call it.
__device__ __forceinline__ void norm_quantize8(const NormArgs& a, const float (&v)[8], bool live, int64_t row,
                                               int64_t col, int64_t nkb, float G, float enc) {
  const int lane = threadIdx.x & 31;
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = fmaxf(amax, live ? fabsf(v[k]) : 0.0f);
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const uint32_t s = block_scale_code(amax, enc);
  const float r = block_inv_scale(s, G);
  uint32_t word = (lane & 1) ? 0u : s << (4 * (lane & 7));
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  if (live) {
    *reinterpret_cast<uint32_t*>(a.q_codes + row * (a.cols >> 1) + (col >> 1)) = r > 0.0f ? block_codes8(v, r) : 0u;
    if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(a.q_sf + sf_word_offset(row, col >> 4, nkb)) = word;
  }
}

// For few rows. One row per CTA (ONE_WARP: per warp); thread t holds the eight columns at 8 t, and with NV > 1
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
    if (a.q_codes != nullptr) norm_quantize8(a, v[i], live[i], row, col[i], nkb, G, enc);
  }
}

namespace normcfg {
constexpr int FWD_MAX_STAGES = 8;
// Rows per CTA from which the ring kernel is taken. Ring against one row per CTA, us (bf16): at 2 rows
// 4096 columns 5.9 / 6.0, 8192 6.0 / 5.2, 1024 6.2 / 6.9; at 2.7 rows 2560 columns 7.4 / 6.0; at 4 rows
// 4096 columns 10.7 / 13.6, 8192 10.8 / 13.4, 1024 11.8 / 15.5.
constexpr int RING_ROWS = 3;
constexpr int SMEM = 220 * 1024;         // per SM, for its CTAs' row buffers and SMEM_OTHER each
constexpr int SMEM_OTHER = 3584;         // a CTA's static and reserved (1 KB) shared memory
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr int GRAD_THREADS = 512;        // threads per SM that the gradient kernel's registers allow
constexpr int GRAD_MAX_STAGES = 8;
constexpr int REDUCE_WARPS = 16;
// Static shared memory: the sums (`floats`), the barriers and what a wait that gave up leaves.
constexpr int smem_static(int floats, int barriers) { return 4 * floats + 8 * barriers + 16; }
constexpr int FWD_RED = 2 * 3 * 16;      // floats for the sums of the ring kernel
__host__ __device__ constexpr int grad_red(bool cluster) { return (cluster ? 4 : 1) * 16 * 8; }  // half the gradient's
static_assert(1024 + smem_static(FWD_RED, FWD_MAX_STAGES + 1) <= SMEM_OTHER, "ring kernel");
static_assert(1024 + smem_static(2 * grad_red(false), GRAD_MAX_STAGES + 1) <= SMEM_OTHER, "gradient");
// Where a cluster shares a row, its sums need more than SMEM_OTHER; a CTA then has its SM to itself (from 4104 columns
// on it has more than GRAD_THREADS / 2 threads), and they lie in what SMEM leaves of the SM's 228 KB and the CTA's 227.
static_assert(SMEM - SMEM_OTHER + 1024 + smem_static(2 * grad_red(true), GRAD_MAX_STAGES + 1) <= 228 * 1024, "");
}  // namespace normcfg

// A sequence's vectors on their way to a CTA's registers: one bulk copy each into shared memory, all in
// flight together. (Loaded straight into registers, each was waited for before the next was asked for,
// and since all CTAs ask for the same lines at the start, that took 8 us of 4096 x 4096's 32.)
struct NormVectors {
  enum { GATE, SCALE, SHIFT, W_POST, W, COUNT };
  uint32_t at[COUNT + 1];  // places in the buffer; absent ones take no room
  __device__ __forceinline__ NormVectors(const void* gate, const void* scale, const void* shift, const void* w_post,
                                         const void* w, int64_t cols, int mod_f32) {
    const void* const p[COUNT] = {gate, scale, shift, w_post, w};
    at[0] = 0u;
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      at[i + 1] = at[i] + (p[i] == nullptr ? 0u : static_cast<uint32_t>(cols * (i >= W_POST || mod_f32 ? 4 : 2)));
  }
  __device__ __forceinline__ uint32_t bytes() const { return at[COUNT]; }
  __device__ __forceinline__ void fetch(int i, uint8_t* buf, const void* p, int64_t first, int mod_f32,
                                        uint64_t* bar) const {  // one thread
    if (at[i + 1] == at[i]) return;
    bulk_load(buf + at[i], static_cast<const char*>(p) + first * (i >= W_POST || mod_f32 ? 4 : 2), at[i + 1] - at[i], bar);
  }
  // Eight values of vector i, or eight times `none`.
  __device__ __forceinline__ void get(int i, const uint8_t* buf, int col, int mod_f32, float none, float (&v)[8]) const {
    if (at[i + 1] == at[i]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = none;
    } else {
      load8_mod(buf + at[i], i >= W_POST || mod_f32, col, v);
    }
  }
};
// Bytes of that buffer.
__host__ __device__ constexpr int64_t norm_vector_bytes(int64_t cols, int mod_f32, int mods, int weights) {
  return cols * (mods * (mod_f32 ? 4 : 2) + weights * 4);
}

__host__ __device__ constexpr int64_t norm_stage(int64_t cols, int elem, bool y) { return cols * (elem + 2 * y); }
// First row of piece g: every piece has `each` rows, the first `extra` one more.
__device__ __forceinline__ int64_t norm_chunk_row(int64_t each, int extra, int g) {
  return each * g + (g < extra ? g : extra);
}

// Warp 0, after its last row, where its wait for row `row` of `rows` gave up (from then on it fetched nothing more):
// the copies that were in flight, of `row` and the rows behind it that the ring holds and of a sequence's vectors,
// are waited for once more, so that none arrives in shared memory that is no longer this CTA's.
__device__ __noinline__ void norm_drain(uint64_t* full, uint64_t* vec_full, uint32_t vec_phase, int row, int64_t rows,
                                        int stages) {
  constexpr uint64_t LIMIT_NS = normcfg::WAIT_LIMIT_NS / 8;
  (void)mbar_wait(vec_full, vec_phase, nullptr, LIMIT_NS, 84);
  for (int r = row; r < row + stages && r < rows; ++r)
    (void)mbar_wait(&full[r % stages], static_cast<uint32_t>(r / stages) & 1u, nullptr, LIMIT_NS, 84);
}

// residual_norm over many rows: a CTA walks a contiguous piece of them. Rows come through a ring of
// row buffers, filled by bulk copies (one per tensor and row, issued by one warp `stages` rows
// ahead), so coming rows are in flight while a row is reduced. A row's first barrier also frees its
// buffer: every thread has read its values by then. Thread t holds the eight columns at 8 (t + i
// threads), i < NV; with NV = 2 the sequence's modulation stays in registers, else it is read again for
// each row (from L1).
// What a row costs beside its elements (barriers, shuffles, the ring) is per warp, so fewer threads
// with more columns each are faster: 4096 x 4096 with NV = 1 and 512 threads took 33.5 us, 7 of them for
// the reductions.
template <class ST, int NV, bool POST>
__global__ void __launch_bounds__(512, 1) residual_norm_ring_kernel(const NormArgs a) {
  using namespace normcfg;
  extern __shared__ __align__(128) uint8_t norm_rows[];
  __shared__ float red[2][3][16];  // FWD_RED
  static_assert(sizeof(red) == 4 * FWD_RED, "");
  __shared__ __align__(8) uint64_t full[FWD_MAX_STAGES], vec_full;
  __shared__ int abort_flag, stuck_row;
  __shared__ uint32_t stuck_vectors;
  griddep_launch_dependents();
  const int g = blockIdx.x;
  const int64_t r0 = norm_chunk_row(a.chunk_rows, a.chunk_extra, g), r1 = norm_chunk_row(a.chunk_rows, a.chunk_extra, g + 1);
  const bool has_y = a.y != nullptr;
  const uint32_t x_bytes = static_cast<uint32_t>(a.cols * sizeof(ST)), y_bytes = has_y ? static_cast<uint32_t>(a.cols * 2) : 0u;
  const uint32_t stage_bytes = x_bytes + y_bytes;
  // Warp 0 fetches a row, one lane per tensor: what a lane copies is set once. (One thread that issued a
  // row's copies one after another held the CTA up: 650 of the gradient's 2600 cycles per row.)
  const int lane = threadIdx.x & 31;
  const uint8_t* const src = static_cast<const uint8_t*>(lane == 0 ? a.x : static_cast<const void*>(a.y));
  const int64_t src_pitch = lane == 0 ? a.ldx * static_cast<int64_t>(sizeof(ST)) : a.ldy * 2;
  const uint32_t src_bytes = lane == 0 ? x_bytes : lane == 1 ? y_bytes : 0u, src_at = lane == 0 ? 0u : x_bytes;
  auto fetch = [&](int64_t row, int stage) {  // warp 0
    if (lane == 0) mbar_arrive_expect_tx(&full[stage], stage_bytes);
    __syncwarp();
    if (src_bytes != 0u) bulk_load(norm_rows + stage * stage_bytes + src_at, src + row * src_pitch, src_bytes, &full[stage]);
  };
  constexpr int NC = NV == 2 ? NV : 1;  // vectors whose modulation is kept
  uint8_t* const vec_buf = norm_rows + a.stages * stage_bytes;
  const NormVectors vecs(a.gate, a.scale, a.shift, POST ? a.w_post : nullptr, a.w, a.cols, a.mod_f32);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
    mbar_init(&vec_full, 1);
    fence_mbarrier_init();
  }
  griddep_wait();  // nothing before this reads or writes global memory
  int64_t b = norm_sequence(a.offsets, a.batches, a.rows_per_batch, r0), seq_end = r0;
  auto fetch_vectors = [&]() {  // one thread
    mbar_arrive_expect_tx(&vec_full, vecs.bytes());
    vecs.fetch(NormVectors::GATE, vec_buf, a.gate, b * a.ldgate, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::SCALE, vec_buf, a.scale, b * a.ldscale, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::SHIFT, vec_buf, a.shift, b * a.ldshift, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::W_POST, vec_buf, a.w_post, 0, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::W, vec_buf, a.w, 0, a.mod_f32, &vec_full);
  };
  if (threadIdx.x < 32) {
    // the vectors before the rows: behind all CTAs' first rows they would take 4 us
    if (threadIdx.x == 0 && NC == NV && b >= 0) fetch_vectors();
    for (int i = 0; i < a.stages && r0 + i < r1; ++i) fetch(r0 + i, i);
  }
  const int64_t nkb = a.cols >> 4;
  if (a.q_codes != nullptr && blockIdx.x == gridDim.x - 1) {  // block scales of the rows that pad to 128 are 0
    const int64_t words = (((a.rows + 127) & ~int64_t(127)) - a.rows) * (a.cols >> 6);
    for (int64_t i = threadIdx.x; i < words; i += blockDim.x)
      *reinterpret_cast<uint32_t*>(a.q_sf + sf_word_offset(a.rows + i / (a.cols >> 6), 4 * (i % (a.cols >> 6)), nkb)) = 0u;
  }
  __syncthreads();

  const float inv_n = 1.0f / static_cast<float>(a.cols);
  bool live[NV];
  int col[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = 8 * static_cast<int>(threadIdx.x + i * blockDim.x);
    live[i] = col[i] < a.cols;
  }
  float G = 0.0f, enc = 0.0f;
  if (a.q_codes != nullptr) {
    G = *a.q_gscale;
    enc = scale_encode_factor(G);
  }
  float cg[NC][8], cs[NC][8], ch[NC][8];  // gate w_post, w (1 + scale), shift
  const int lane16 = threadIdx.x & 15, warps = blockDim.x >> 5;
  auto warp_columns = [&](int w) {  // columns that warp w holds
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = static_cast<int>(a.cols) - 8 * (32 * w + i * static_cast<int>(blockDim.x));
      n += left < 0 ? 0 : left < 256 ? left : 256;
    }
    return w < warps ? static_cast<float>(n) : 0.0f;
  };
  const float my_columns = warp_columns(threadIdx.x >> 5), its_columns = warp_columns(lane16);
  const float my_inv = my_columns > 0.0f ? 1.0f / my_columns : 0.0f;
  auto join = [&](float v) {  // sum over the lanes of a half-warp
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  // Sum over the CTA (at most 16 warps), one barrier.
  auto cta_sum = [&](float v, float* rd) {
    v = row_sum<true>(v, nullptr);
    if ((threadIdx.x & 31) == 0) rd[threadIdx.x >> 5] = v;
    __syncthreads();
    return join(lane16 < warps ? rd[lane16] : 0.0f);
  };
  // gate w_post, w (1 + scale) and shift of vector i, from the buffer (NV = 2) or from global memory
  auto times = [](float (&v)[8], const float (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= w[k];
  };
  auto plus1 = [](float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += 1.0f;
  };
  auto from_buffer = [&](int i, float (&c_g)[8], float (&c_s)[8], float (&c_h)[8]) {
    float w[8];
    vecs.get(NormVectors::GATE, vec_buf, col[i], a.mod_f32, 1.0f, c_g);
    vecs.get(NormVectors::W_POST, vec_buf, col[i], a.mod_f32, 1.0f, w);
    times(c_g, w);
    vecs.get(NormVectors::SCALE, vec_buf, col[i], a.mod_f32, 0.0f, c_s);
    plus1(c_s);
    vecs.get(NormVectors::W, vec_buf, col[i], a.mod_f32, 1.0f, w);
    times(c_s, w);
    vecs.get(NormVectors::SHIFT, vec_buf, col[i], a.mod_f32, 0.0f, c_h);
  };
  auto constants_gate = [&](int i, float (&c_g)[8]) {
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) c_g[k] = 1.0f;
    if (a.gate != nullptr) load8_mod(a.gate, a.mod_f32, b * a.ldgate + col[i], c_g);
    if (POST && a.w_post != nullptr) {
      load8_f32(a.w_post + col[i], w);
      times(c_g, w);
    }
  };
  auto constants_norm = [&](int i, float (&c_s)[8], float (&c_h)[8]) {
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) c_s[k] = c_h[k] = 0.0f;
    if (a.scale != nullptr) load8_mod(a.scale, a.mod_f32, b * a.ldscale + col[i], c_s);
    plus1(c_s);
    if (a.w != nullptr) {
      load8_f32(a.w + col[i], w);
      times(c_s, w);
    }
    if (a.shift != nullptr) load8_mod(a.shift, a.mod_f32, b * a.ldshift + col[i], c_h);
  };

  int stage = 0;
  uint32_t phase = 0u, vec_phase = 0u;
  bool arrives = true;  // no wait of warp 0 has given up
  auto fetch_next = [&](int64_t row, bool in_time) {  // warp 0, once the buffer of `row` is free
    if (!__all_sync(0xffffffffu, in_time || !arrives)) {
      arrives = false;
      stuck_row = static_cast<int>(row - r0);
      stuck_vectors = vec_phase ^ 1u;  // of the vectors that were waited for last
    }
    if (arrives && row + a.stages < r1) fetch(row + a.stages, stage);
  };
  for (int64_t row = r0; row < r1; ++row) {
    bool in_time = true;
    if (row >= seq_end) {
      if (row != r0) b = norm_sequence(a.offsets, a.batches, a.rows_per_batch, row);
      if (b < 0) {  // rows without a sequence are left as they are
        seq_end = row + 1;
      } else {
        seq_end = a.offsets == nullptr ? (b + 1) * a.rows_per_batch : static_cast<int64_t>(a.offsets[b + 1]);
        if constexpr (NC == NV) {
          // a barrier lies behind since the last sequence's were read
          if (threadIdx.x == 0 && row != r0 && arrives) fetch_vectors();
          in_time = mbar_wait(&vec_full, vec_phase, &abort_flag, WAIT_LIMIT_NS, 82);
          vec_phase ^= 1u;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (live[i]) from_buffer(i, cg[i], cs[i], ch[i]);
          }
        }
      }
    }
    in_time = mbar_wait(&full[stage], phase, &abort_flag, WAIT_LIMIT_NS, 81) && in_time;
    const uint8_t* buf = norm_rows + stage * stage_bytes;
    bool freed = false;  // a barrier has been passed since the row's values were read
    auto refill = [&]() {
      if (!freed && threadIdx.x < 32) fetch_next(row, in_time);
      freed = true;
    };
    if (b >= 0) {
      float (*rd)[16] = red[static_cast<int>(row - r0) & 1];
      float v[NV][8];
      Stream8<uint16_t> ys[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live[i]) continue;
        Stream8<ST> xs;
        xs.load(buf, col[i]);
        xs.get(v[i]);
        if (has_y) ys[i].load(buf + x_bytes, col[i]);
      }
      float rstd_y = 1.0f;
      if constexpr (POST) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!live[i]) continue;
          float yv[8];
          ys[i].get(yv);
#pragma unroll
          for (int k = 0; k < 8; ++k) ss = fmaf(yv[k], yv[k], ss);
        }
        rstd_y = rsqrtf(cta_sum(ss, rd[0]) * inv_n + a.eps);
        refill();
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live[i]) continue;
        constexpr bool again = NC != NV;
        if constexpr (again) constants_gate(i, cg[0]);
        Stream8<ST> xs;
        if (has_y) {
          float yv[8];
          ys[i].get(yv);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if constexpr (POST) yv[k] *= rstd_y;
            v[i][k] = fmaf(a.alpha, v[i][k], yv[k] * cg[again ? 0 : i][k]);
          }
        }
        xs.round(v[i]);
        if (a.x_out != nullptr) xs.store(a.x_out, row * a.ldxo + col[i]);
      }
      float mean = 0.0f, rstd = 1.0f;
      if (a.norm == NORM_LAYER) {
        // Each warp's mean and centred sum of squares, then (after one barrier) those of the row:
        // sum of squares about the row's mean = sum over warps of (theirs + n (their mean - mean)^2).
        // As exact as a second pass over the values.
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!live[i]) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k) sum += v[i][k];
        }
        const float wmean = row_sum<true>(sum, nullptr) * my_inv;
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!live[i]) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float d = v[i][k] - wmean;
            ss = fmaf(d, d, ss);
          }
        }
        ss = row_sum<true>(ss, nullptr);
        if ((threadIdx.x & 31) == 0) {
          rd[1][threadIdx.x >> 5] = wmean;
          rd[2][threadIdx.x >> 5] = ss;
        }
        __syncthreads();
        const float m = lane16 < warps ? rd[1][lane16] : 0.0f, q = lane16 < warps ? rd[2][lane16] : 0.0f;
        mean = join(its_columns * m) * inv_n;
        rstd = rsqrtf(join(fmaf(its_columns * (m - mean), m - mean, q)) * inv_n + a.eps);
        refill();
      } else if (a.norm == NORM_RMS) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!live[i]) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
        }
        rstd = rsqrtf(cta_sum(ss, rd[2]) * inv_n + a.eps);
        refill();
      }
      if (a.stats != nullptr && threadIdx.x == 0)
        *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(mean, rstd, rstd_y, 0.0f);
      if (a.norm != NORM_NONE) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          Stream8<uint16_t> out;
          out.q = make_uint4(0u, 0u, 0u, 0u);
          if (live[i]) {
            constexpr bool again = NC != NV;
            if constexpr (again) constants_norm(i, cs[0], ch[0]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[i][k] = fmaf((v[i][k] - mean) * rstd, cs[again ? 0 : i][k], ch[again ? 0 : i][k]);
            out.round(v[i]);
            if (a.h != nullptr) out.store(a.h, row * a.ldh + col[i]);
          }
          if (a.q_codes != nullptr) norm_quantize8(a, v[i], live[i], row, col[i], nkb, G, enc);
        }
      }
    }
    if (!freed) __syncthreads();
    refill();
    if (++stage == a.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (!arrives) norm_drain(full, &vec_full, stuck_vectors, stuck_row, r1 - r0, a.stages);
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
// Rows are cut into `chunks` contiguous pieces, one CTA or cluster each; a thread keeps its columns and
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
  int chunks, stages;     // pieces of the rows, row buffers
  int cluster, cta_cols;  // CTAs that share a row, and the columns of each
  int64_t chunk_rows;     // rows of a piece, and how many pieces have one more
  int chunk_extra;
  float* seq_part;        // (chunks + batches) x 3 x cols, or null (no sums)
  float* w_part;          // chunks x 2 x cols, or null (neither dw nor dw_post)
  int* seq_pieces;        // batches x 2: the first and the last piece that hold rows of a sequence
};

// Bytes of one row's buffer: the stream, its gradient, the gradient of h, the branch, the statistics
// (absent ones take no room).
__host__ __device__ constexpr int64_t norm_grad_stage(int64_t cols, int elem, bool dxo, bool dh, bool y) {
  return cols * (elem * (dxo + dh) + 2 * (dh + y)) + 16;
}

// Sums over the CTA, or over a cluster that shares the row's columns, of the first N of six values per
// thread (N = 2 or 6); every thread gets them. Within a warp, each of the first log2 exchanges halves
// the values a lane keeps (9 shuffles for six sums instead of 30); lane 4 k then holds sum k. `red` holds
// 32 x 8 floats; in a cluster each warp writes its sums to that place in every CTA, and the cluster's
// barrier takes the place of the CTA's.
template <int N, bool CLUSTER>
__device__ __forceinline__ void row_sums(float (&s)[6], float* red, int rank, int cluster) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float v;
  bool holds;
  int at;
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
    holds = (lane & 3) == 0;
    at = lane >> 2;
  } else {
    const bool h16 = (lane & 16) != 0;
    v = (h16 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, h16 ? s[0] : s[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    holds = (lane & 15) == 0;
    at = lane >> 4;
  }
  int entries = warps;
  if constexpr (CLUSTER) {
    entries = cluster * warps;
    const uint32_t mine = smem_u32(red + (rank * warps + warp) * 8 + at);
    if (holds) {
      for (int c = 0; c < cluster; ++c)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(mine, c)), "f"(v) : "memory");
    }
    cluster_sync_all();
  } else {
    if (holds) red[warp * 8 + at] = v;
    __syncthreads();
  }
  v = 0.0f;
  for (int w = lane >> 3; w < entries; w += 4) v += red[w * 8 + (lane & 7)];
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = __shfl_sync(0xffffffffu, v, k);
}

// A CTA walks the rows of its piece; thread t holds eight columns. Rows come through a ring of row
// buffers, filled by bulk copies (one per tensor and row, issued by one warp `stages` rows ahead), so the
// loads of the coming rows are in flight while a row is reduced. The one barrier of a row's reduction is
// also what frees its buffer: every thread has read its values by then.
// POST: the branch has its norm (six row sums, else two).
// CLUSTER: above 4096 columns the CTAs of a cluster of 2 or 4 share a row's columns, so that a thread's
// sums and the sequence's vectors still fit in its registers (with 16 columns per thread, spilling and
// reading the vectors again for each row, 8192 x 5120 took 291 us).
template <class ST, bool POST, bool CLUSTER>
__global__ void __launch_bounds__(normcfg::GRAD_THREADS, 1) residual_norm_grad_kernel(const NormGradArgs a) {
  using namespace normcfg;
  extern __shared__ __align__(128) uint8_t norm_rows[];
  __shared__ float red[2][grad_red(CLUSTER)];
  __shared__ __align__(8) uint64_t full[GRAD_MAX_STAGES], vec_full;
  __shared__ int abort_flag, stuck_row;
  __shared__ uint32_t stuck_vectors;
  griddep_launch_dependents();
  constexpr int NV = 1;
  const int cluster = CLUSTER ? a.cluster : 1;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0, g = static_cast<int>(blockIdx.x) / cluster;
  const int col0 = rank * a.cta_cols;  // this CTA's columns
  const int ncols = static_cast<int>(a.cols) - col0 < a.cta_cols ? static_cast<int>(a.cols) - col0 : a.cta_cols;
  const int64_t r0 = norm_chunk_row(a.chunk_rows, a.chunk_extra, g), r1 = norm_chunk_row(a.chunk_rows, a.chunk_extra, g + 1);
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  const bool has_dxo = a.dxo != nullptr, has_dh = a.dh != nullptr, has_y = a.y != nullptr;
  // the parts of a row buffer
  const uint32_t stream_bytes = static_cast<uint32_t>(ncols * sizeof(ST)), half_bytes = static_cast<uint32_t>(ncols * 2);
  const uint32_t at_dxo = has_dh ? stream_bytes : 0u, at_dh = at_dxo + (has_dxo ? stream_bytes : 0u);
  const uint32_t at_y = at_dh + (has_dh ? half_bytes : 0u), at_stats = at_y + (has_y ? half_bytes : 0u);
  const uint32_t stage_bytes = at_stats + 16u;

  // warp 0 fetches a row, one lane per tensor
  const int lane = threadIdx.x & 31;
  const void* const src_of[5] = {a.x, a.dh, a.dxo, a.y, a.stats};
  const int64_t pitch_of[5] = {a.ldx * static_cast<int64_t>(sizeof(ST)), a.lddh * 2,
                               a.lddxo * static_cast<int64_t>(sizeof(ST)), a.ldy * 2, 16};
  const uint32_t bytes_of[5] = {has_dh ? stream_bytes : 0u, has_dh ? half_bytes : 0u, has_dxo ? stream_bytes : 0u,
                                has_y ? half_bytes : 0u, 16u};
  const uint32_t at_of[5] = {0u, at_dh, at_dxo, at_y, at_stats};
  const uint8_t* src = nullptr;
  int64_t src_pitch = 0;
  uint32_t src_bytes = 0u, src_at = 0u;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    if (lane != i) continue;
    src = static_cast<const uint8_t*>(src_of[i]) + (i == 4 ? 0 : col0 * (i == 0 || i == 2 ? static_cast<int>(sizeof(ST)) : 2));
    src_pitch = pitch_of[i];
    src_bytes = bytes_of[i];
    src_at = at_of[i];
  }
  auto fetch = [&](int64_t row, int stage) {  // warp 0
    if (lane == 0) mbar_arrive_expect_tx(&full[stage], stage_bytes);
    __syncwarp();
    if (src_bytes != 0u) bulk_load(norm_rows + stage * stage_bytes + src_at, src + row * src_pitch, src_bytes, &full[stage]);
  };
  uint8_t* const vec_buf = norm_rows + a.stages * stage_bytes;
  const NormVectors vecs(a.gate, a.scale, nullptr, POST ? a.w_post : nullptr, a.w, ncols, a.mod_f32);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
    mbar_init(&vec_full, 1);
    fence_mbarrier_init();
  }
  griddep_wait();  // nothing before this reads or writes global memory
  int64_t b = norm_sequence(a.offsets, a.batches, a.rows_per_batch, r0), seq_end = r0;
  auto fetch_vectors = [&]() {  // one thread
    mbar_arrive_expect_tx(&vec_full, vecs.bytes());
    vecs.fetch(NormVectors::GATE, vec_buf, a.gate, b * a.ldgate + col0, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::SCALE, vec_buf, a.scale, b * a.ldscale + col0, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::W_POST, vec_buf, a.w_post, col0, a.mod_f32, &vec_full);
    vecs.fetch(NormVectors::W, vec_buf, a.w, col0, a.mod_f32, &vec_full);
  };
  if (threadIdx.x < 32) {
    // the vectors before the rows: behind all CTAs' first rows they would take 4 us
    if (threadIdx.x == 0 && b >= 0) fetch_vectors();
    for (int i = 0; i < a.stages && r0 + i < r1; ++i) fetch(r0 + i, i);
  }
  __syncthreads();
  if constexpr (CLUSTER) cluster_sync_all();  // every CTA of the cluster has started

  bool live[NV];
  int col[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = 8 * static_cast<int>(threadIdx.x + i * blockDim.x);
    live[i] = col[i] < ncols;
  }
  float s_dh[NV][8], s_dhx[NV][8], s_ty[NV][8];  // sums over the current sequence's rows
  float c_w[NV][8], c_g[NV][8], c_a[NV][8];  // w (1 + scale), the gate, gate w_post
  bool first_flush = true, seq_begins = false;

  auto flush = [&](int64_t next_row) {
    if (a.seq_part == nullptr) return;  // no sums are asked for
    if (threadIdx.x == 0 && rank == 0) {
      if (seq_begins) a.seq_pieces[2 * b] = g;
      if (next_row >= seq_end || next_row >= a.rows) a.seq_pieces[2 * b + 1] = g;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      const int at = col0 + col[i];
      float* p = a.seq_part + (g + b) * 3 * a.cols + at;
      store8_f32(p, s_dh[i]);
      store8_f32(p + a.cols, s_dhx[i]);
      store8_f32(p + 2 * a.cols, s_ty[i]);
      if (a.w_part != nullptr) {
        float* q = a.w_part + static_cast<int64_t>(g) * 2 * a.cols + at;
        float w0[8], p0[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w0[k] = 0.0f, p0[k] = 1.0f;
        if (a.scale != nullptr) load8_mod(a.scale, a.mod_f32, b * a.ldscale + at, w0);
        if (a.gate != nullptr) load8_mod(a.gate, a.mod_f32, b * a.ldgate + at, p0);
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
  uint32_t phase = 0u, vec_phase = 0u;
  bool arrives = true;  // no wait of warp 0 has given up
  auto fetch_next = [&](int64_t row, bool in_time) {  // warp 0, once the buffer of `row` is free
    if (!__all_sync(0xffffffffu, in_time || !arrives)) {
      arrives = false;
      stuck_row = static_cast<int>(row - r0);
      stuck_vectors = vec_phase ^ 1u;  // of the vectors that were waited for last
    }
    if (arrives && row + a.stages < r1) fetch(row + a.stages, stage);
  };
  for (int64_t row = r0; row < r1; ++row) {
    bool skip = false, in_time = true;
    if (row >= seq_end) {
      if (row != r0) {
        if (b >= 0) flush(row);
        b = norm_sequence(a.offsets, a.batches, a.rows_per_batch, row);
      }
      if (b < 0) {  // rows without a sequence are left as they are
        seq_end = row + 1;
        skip = true;
      } else {
        seq_end = a.offsets == nullptr ? (b + 1) * a.rows_per_batch : static_cast<int64_t>(a.offsets[b + 1]);
        seq_begins = row == (a.offsets == nullptr ? b * a.rows_per_batch : static_cast<int64_t>(a.offsets[b])) || row == 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int k = 0; k < 8; ++k) s_dh[i][k] = s_dhx[i][k] = s_ty[i][k] = 0.0f;
        }
        {
          // a barrier lies behind since the last sequence's were read
          if (threadIdx.x == 0 && row != r0 && arrives) fetch_vectors();
          in_time = mbar_wait(&vec_full, vec_phase, &abort_flag, WAIT_LIMIT_NS, 83);
          vec_phase ^= 1u;
          if (live[0]) {
            float v[8];
            vecs.get(NormVectors::SCALE, vec_buf, col[0], a.mod_f32, 0.0f, c_w[0]);
            vecs.get(NormVectors::W, vec_buf, col[0], a.mod_f32, 1.0f, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) c_w[0][k] = (1.0f + c_w[0][k]) * v[k];
            vecs.get(NormVectors::GATE, vec_buf, col[0], a.mod_f32, 1.0f, c_g[0]);
            vecs.get(NormVectors::W_POST, vec_buf, col[0], a.mod_f32, 1.0f, c_a[0]);
#pragma unroll
            for (int k = 0; k < 8; ++k) c_a[0][k] *= c_g[0][k];
          }
        }
      }
    }
    in_time = mbar_wait(&full[stage], phase, &abort_flag, WAIT_LIMIT_NS, 80) && in_time;
    const uint8_t* buf = norm_rows + stage * stage_bytes;
    if (skip) {
      if constexpr (CLUSTER) {
        cluster_sync_all();
      } else {
        __syncthreads();
      }
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
      row_sums<POST ? 6 : 2, CLUSTER>(s, red[static_cast<int>(row - r0) & 1], rank, cluster);
      if (!CLUSTER && threadIdx.x < 32) fetch_next(row, in_time);
      const float m1 = a.norm == NORM_LAYER ? s[0] * inv_n : 0.0f, m2 = s[1] * inv_n;
      const float m3 = POST ? (s[2] + rstd * (s[3] - m1 * s[4] - m2 * s[5])) * inv_n : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live[i]) continue;
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
          v.store(a.dx, row * a.lddx + col0 + col[i]);
        }
        if (a.dy != nullptr) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = POST ? rstd_y * (c_a[0][k] * t[i][k] - yh[i][k] * m3) : c_g[0][k] * t[i][k];
          Stream8<uint16_t> v;
          v.round(o);
          v.store(a.dy, row * a.lddy + col0 + col[i]);
        }
      }
    }
    // Every thread has passed this row's barrier, so its buffer takes the next row. (A CTA with whole rows asks for it
    // right behind the barrier, a cluster's here: 16384 x 4096 153 and 157 us, 8192 x 5120 203 and 193 us.)
    if ((CLUSTER || skip) && threadIdx.x < 32) fetch_next(row, in_time);
    if (++stage == a.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (b >= 0) flush(r1);
  if (a.w_part != nullptr && first_flush) {  // none of this piece's rows has a sequence
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      for (int k = 0; k < 8; ++k) {
        a.w_part[static_cast<int64_t>(g) * 2 * a.cols + col0 + col[i] + k] = 0.0f;
        a.w_part[(static_cast<int64_t>(g) * 2 + 1) * a.cols + col0 + col[i] + k] = 0.0f;
      }
    }
  }
  if (!arrives) norm_drain(full, &vec_full, stuck_vectors, stuck_row, r1 - r0, a.stages);
  if constexpr (CLUSTER) cluster_sync_all();  // no CTA leaves while another may write its sums there
}

// Adds up the slots of each sequence and the pieces' weight sums. Block (x, y): columns 32 x and
// on; y < gridDim.y - 1 takes the sequences y, y + gridDim.y - 1, ..., the last y the weights.
// 16 warps share the slots, one column per lane, and are joined in a fixed order (a half-warp then adds
// a column over the warps). With 148 to 2368 pieces (74 or 32 where a cluster shares a row;
// never more than rows) the kernel is bound by the latency of a thread's loads one after another, and by how
// many blocks fit at once (32 warps at 64 registers: one per SM, five waves at 4096 columns and 4 sequences).
// Loads past the end are left out one by one: in a loop unrolled as it is, the remainder's wait for one
// another (1536 x 2048 with 16 sequences and the weights' sums: 25.9 -> 23.5 us for the whole gradient).
// PER_SM: with 4 blocks per SM a thread has 32 registers, with 2 it has more loads in flight. 2 where all blocks
// fit at once (1531 x 2048, 3 sequences: 21.6 -> 19.5 us; 16 sequences: 23.5 -> 25.5 us).
template <int PER_SM>
__global__ void __launch_bounds__(32 * normcfg::REDUCE_WARPS, PER_SM) norm_grad_reduce_kernel(const NormGradArgs a) {
  using normcfg::REDUCE_WARPS;
  __shared__ float red[3][REDUCE_WARPS][33];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = 2 * warp + (lane >> 4);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;        // while adding slots
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + mine;        // while joining
  const bool live = col < a.cols, last = (lane & 15) == 0 && out < a.cols;
  griddep_wait();
  auto total = [&](int k) {
    float v = red[k][lane & 15][mine];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  if (blockIdx.y == gridDim.y - 1) {
    float s0 = 0.0f, s1 = 0.0f;
    if (live && a.w_part != nullptr) {
      const float* p = a.w_part + static_cast<int64_t>(warp) * 2 * a.cols + col;
      constexpr int U = 7;
      for (int g = warp; g < a.chunks; g += U * REDUCE_WARPS) {
        float u[U][2];
#pragma unroll
        for (int i = 0; i < U; ++i, p += 2 * REDUCE_WARPS * a.cols) {
          const bool in = g + i * REDUCE_WARPS < a.chunks;
          u[i][0] = in ? p[0] : 0.0f;
          u[i][1] = in ? p[a.cols] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          s0 += u[i][0];
          s1 += u[i][1];
        }
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
    // unchecked offsets may leave these unwritten: kept in range
    int g0 = a.seq_pieces[2 * b], g1 = a.seq_pieces[2 * b + 1];
    g0 = g0 < 0 ? 0 : g0 < a.chunks ? g0 : a.chunks - 1;
    g1 = g1 < a.chunks ? g1 : a.chunks - 1;
    float v[3] = {0.0f, 0.0f, 0.0f};
    if (s < e) {
      if (live) {
        const float* p = a.seq_part + (g0 + warp + b) * 3 * a.cols + col;
        constexpr int U = PER_SM == 2 ? 7 : 4;
        for (int g = g0 + warp; g <= g1; g += U * REDUCE_WARPS) {
          float u[U][3];
#pragma unroll
          for (int i = 0; i < U; ++i, p += 3 * REDUCE_WARPS * a.cols) {
            const bool in = g + i * REDUCE_WARPS <= g1;
            u[i][0] = in ? p[0] : 0.0f;
            u[i][1] = in ? p[a.cols] : 0.0f;
            u[i][2] = in ? p[2 * a.cols] : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int k = 0; k < 3; ++k) v[k] += u[i][k];
          }
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
