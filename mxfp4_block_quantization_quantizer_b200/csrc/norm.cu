// Layer norm in front of a quantized linear layer, and its gradients
// (sm_100a).
//
// Forward, per row of x [rows][cols]:
//   mean = sum(x) / cols,  var = sum((x - mean)^2) / cols,
//   rstd = (var + eps)^-1/2,  y = (x - mean) rstd w + b
// and, fused, the 1x32 nearest-even quantization of the rounded y.
// Backward, with h = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean_c(g) - h mean_c(g h)),
//   dw = sum_r dy h,  db = sum_r dy.
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and
// writes dx, once each. W warps take whole rows (E = VEC NV elements a thread
// in registers; rows too wide for one CTA are split over a cluster of two).
// The loads of the next rows (ln_depth) are in flight at any time as 16-byte
// asynchronous copies into shared memory: each thread copies what it will
// read itself, so no barrier orders them, and no register holds them. Every
// statistic is fp32: each warp takes its own mean first and sums squares
// around it, and the warps' pairs (sum, squares) are joined with the exact
// correction n_w (mean_w - mean)^2, so the variance of data far from zero does
// not cancel (the mean itself has the error of an fp32 sum, some 2^-24 of the
// row's mean |x|, which reaches y times rstd w). Persistent grid: the warps keep their columns from row to row,
// so w and b stay in registers, and so do the column sums of the backward
// pass; each CTA writes one partial row of dw and db and a second small
// kernel adds those in a fixed order (no atomics: the same inputs give the
// same bits).
//
// Rows that are no whole number of 16-byte vectors start off a 16-byte
// boundary, each at its own distance `off`; but rows VEC apart start at the
// same distance, so with a row stride between a group's rows that is a
// multiple of VEC a thread still keeps its columns, and everything but the
// two ends of a row moves as aligned 16-byte vectors (vectors that reach into
// a neighbouring row are read whole and masked, and stored element by
// element).
//
// Measured, of a plain copy's rate: forward 12608 x 1536 bf16 15.2 us (78%),
// 8192 x 4096 bf16 25.5 us (81%), 4096 x 14336 fp32 86 us (83%), 5000 x 2563
// bf16 (off the boundary) 21.5 us (36%), with the quantization 12608 x 1536
// bf16 20.7 us (36%; y too: 21.3 us, 63%); backward 12608 x 1536 bf16 28.4 us
// (63%), 8192 x 4096 bf16 44.7 us (69%), 4096 x 14336 fp32 158 us (68%).
#include "launch.cuh"
#include "mxfp4_device.cuh"

namespace mxfp4 {

namespace {

constexpr int kLnMaxWarps = 16;      // warps of a CTA that share a row
constexpr int kLnMaxParts = 32;      // ... and of a cluster
// Rows in flight per group.
__host__ __device__ constexpr int ln_depth(int nv) { return nv == 1 ? 4 : 2; }
// Warps of a CTA that narrow rows share (backward: few partial sums).
constexpr int kLnFwdWarps = 4, kLnBwdWarps = 16;
// The backward kernel that takes several rows at a time: most warps of a row,
// and warps and row groups of a CTA that narrow rows share.
constexpr int kLnRowWarps = 16, kLnRowShare = 12, kLnRowGroups = 6;
constexpr int64_t kLnMaxCols = 1 << 16;  // far above what a cluster holds
constexpr int kLnGenThreads = 512;   // the kernels for wider rows
constexpr int kLnRedThreads = 1024;

// Two fp32 values per instruction (sm_100a's packed fp32 arithmetic).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float f2_lo(F2 a) {
  return __uint_as_float(static_cast<uint32_t>(a.v));
}
__device__ __forceinline__ float f2_hi(F2 a) {
  return __uint_as_float(static_cast<uint32_t>(a.v >> 32));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A vector of VEC elements as loaded (16 bytes), and its fp32 pairs.
template <bool BF16, int VEC>
struct Vec;
template <>
struct Vec<true, 8> {
  uint4 r;
  __device__ __forceinline__ void unpack(F2* p) const {
    p[0] = f2(bf16_lo(r.x), bf16_hi(r.x)), p[1] = f2(bf16_lo(r.y), bf16_hi(r.y));
    p[2] = f2(bf16_lo(r.z), bf16_hi(r.z)), p[3] = f2(bf16_lo(r.w), bf16_hi(r.w));
  }
  __device__ __forceinline__ void pack(const F2* p) {
    r = make_uint4(pack_bf16x2(f2_lo(p[0]), f2_hi(p[0])), pack_bf16x2(f2_lo(p[1]), f2_hi(p[1])),
                   pack_bf16x2(f2_lo(p[2]), f2_hi(p[2])), pack_bf16x2(f2_lo(p[3]), f2_hi(p[3])));
  }
};
template <>
struct Vec<false, 4> {
  uint4 r;
  __device__ __forceinline__ void unpack(F2* p) const {
    p[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
    p[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  __device__ __forceinline__ void pack(const F2* p) {
    r = make_uint4(__float_as_uint(f2_lo(p[0])), __float_as_uint(f2_hi(p[0])),
                   __float_as_uint(f2_lo(p[1])), __float_as_uint(f2_hi(p[1])));
  }
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
// Sum over lanes 0 .. P - 1 (P a power of two), for every lane of a warp
// whose lanes from P on repeat lanes l % P.
__device__ __forceinline__ float part_sum(float v, int P) {
  for (int o = P >> 1; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Sums of two values over a warp with one shuffle more than for one: lane 0
// gets a's (and every lane of the lower half), lane 16 b's.
__device__ __forceinline__ float warp_sum2(float a, float b, int lane) {
  const bool up = (lane & 16) != 0;
  float v = __fadd_rn(up ? b : a, __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, 16));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// v^-1/2 to an ulp: the approximation and one Newton step.
__device__ __forceinline__ float rsqrt_exact(float v) {
  const float r = rsqrtf(v);
  const float e = __fmaf_rn(-__fmul_rn(v, r), r, 1.0f);
  const float n = __fmaf_rn(__fmul_rn(0.5f, r), e, r);
  return v > 0.0f && v < __uint_as_float(0x7F800000u) ? n : r;
}

// Barrier of the W > 1 warps of row group g, of at most MAXG in the CTA. (With
// the barrier's number in a register a CTA reserves all 16, and four CTAs all
// of an SM's.)
template <int MAXG>
__device__ __forceinline__ void group_sync(int g, int W) {
  if (g == MAXG - 1)
    asm volatile("bar.sync %0, %1;" ::"n"(MAXG), "r"(W * 32) : "memory");
  else if constexpr (MAXG > 1)
    group_sync<MAXG - 1>(g, W);
}
// Every thread of both CTAs of a cluster (release, then acquire).
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A cluster's CTAs may start at different times, and none may be written to
// before it runs: every thread arrives as its kernel begins and waits before
// the first row, when the loads ahead of that are under way.
__device__ __forceinline__ void pair_started() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_wait_started() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_pair(float2* p, float2 v, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y)
               : "memory");
}

// How rows are shared out: W warps of a CTA (times CS CTAs of a cluster) take
// a row, G groups a CTA; P = the power of two from W CS on.
struct LnSplit {
  int W, P, CS, G;
};

// Where a thread stands. Its vectors are v0, v0 + 32, ... of the row's nvec,
// which starts `off` elements after a 16-byte boundary. Its group takes `n`
// rows: row0, row0 + stride, ...; where rows may start off the boundary
// (EDGE), a CTA keeps to rows that are equal modulo VEC, which all start at
// one `off`.
struct Place {
  int W, CS, P, g, w, lane, rank, warp, v0, off, nvec, cols, n;
  int64_t row0, stride;
};
template <int VEC, int NV, bool EDGE>
__device__ __forceinline__ Place place(const LnSplit& s, int64_t rows, int cols, int64_t ld,
                                       int misaligned) {
  Place p;
  p.W = s.W, p.CS = s.CS, p.P = s.P, p.cols = cols;
  p.warp = threadIdx.x >> 5;
  p.g = p.warp / s.W, p.w = p.warp % s.W, p.lane = threadIdx.x & 31;
  p.rank = s.CS > 1 ? int(blockIdx.x & 1) : 0;
  p.v0 = (p.rank * s.W + p.w) * NV * 32 + p.lane;
  const int64_t b = blockIdx.x / s.CS, nb = gridDim.x / s.CS;
  if constexpr (EDGE) {
    p.row0 = b % VEC + ((b / VEC) * s.G + p.g) * VEC;
    p.stride = nb * s.G;  // nb is a multiple of VEC
  } else {
    p.row0 = b * s.G + p.g;
    p.stride = nb * s.G;
  }
  p.n = p.row0 < rows ? int((rows - p.row0 + p.stride - 1) / p.stride) : 0;
  p.off = EDGE ? int((misaligned + (b % VEC) * ld) & (VEC - 1)) : 0;
  p.nvec = (cols + p.off + VEC - 1) / VEC;
  return p;
}
// Elements of the row that warp `part` (of W CS) holds.
template <int VEC, int NV>
__device__ __forceinline__ float part_count(const Place& p, int part) {
  const int e = part * NV * 32 * VEC - p.off;
  return float(min(max(e + NV * 32 * VEC, 0), p.cols) - min(max(e, 0), p.cols));
}

// Starts the copy of the vector at `src` into dst. EDGE: the vectors at the
// tensor's two ends may reach past it and are cut.
template <bool BF16, bool EDGE>
__device__ __forceinline__ void fetch_vec(uint4* dst, const uint8_t* src, const uint8_t* first,
                                          const uint8_t* end) {
  if (EDGE && src < first) {
    // ahead of the first element: single elements, by plain loads
    uint32_t w[4] = {0, 0, 0, 0};
    for (int b = int(first - src); b < 16; b += BF16 ? 2 : 4) {
      if (src + b >= end) break;
      if constexpr (BF16)
        w[b / 4] |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(src + b))) << (8 * (b & 2));
      else
        w[b / 4] = __ldg(reinterpret_cast<const uint32_t*>(src + b));
    }
    *dst = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (EDGE && end - src < 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(dst)),
                 "l"(src), "r"(int(end - src))
                 : "memory");
  } else {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
  }
}

// A thread's way down the rows of one input: `at` is its first vector in the
// next row to load, [first, end) the tensor.
struct Walk {
  const uint8_t *at, *first, *end;
  int64_t step;  // bytes from a row of the group to its next
};
template <bool BF16>
__device__ __forceinline__ Walk walk(const void* base, int64_t rows, int64_t ld, const Place& p) {
  constexpr int kSize = BF16 ? 2 : 4, VEC = 16 / kSize;
  Walk w;
  w.first = static_cast<const uint8_t*>(base);
  w.end = w.first + ((rows - 1) * ld + p.cols) * kSize;
  w.at = w.first + (p.row0 * ld + int64_t(p.v0) * VEC - p.off) * kSize;
  w.step = p.stride * ld * kSize;
  return w;
}
// Rows at either end of a tensor whose vectors may reach past it.
template <int VEC>
__device__ __forceinline__ int64_t end_rows(int64_t ld) {
  return ld > VEC ? 1 : VEC / int(ld) + 1;
}

// A parameter (fp32 [cols], nullptr: `fill`) of this CTA's vectors in shared
// memory: [VEC / 4][slots] float4, slot s = vector rank W NV 32 + s (so that
// a warp's 16-byte reads touch every bank once); asynchronous copies. Outside the row:
// zero, or `fill` (nothing there is stored).
template <int VEC, int NV, bool EDGE>
__device__ __forceinline__ void stage_param(const float* param, float fill, const Place& p,
                                            float* to) {
  const int slots = p.W * NV * 32, base = p.rank * slots * VEC - p.off;
  if (param == nullptr) {
    for (int i = threadIdx.x; i < slots * VEC; i += blockDim.x) to[i] = fill;
  } else if (EDGE || (reinterpret_cast<uintptr_t>(param) & 15u) != 0) {
    for (int i = threadIdx.x; i < slots * VEC; i += blockDim.x) {
      const int c = base + i, s = i / VEC, j = i % VEC;
      const bool in = c >= 0 && c < p.cols;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(
                       smem_addr(to + (j / 4 * slots + s) * 4 + j % 4)),
                   "l"(param + (in ? c : 0)), "r"(in ? 4 : 0)
                   : "memory");
    }
  } else {
    for (int i = threadIdx.x; i < slots * (VEC / 4); i += blockDim.x) {
      const int c = base + 4 * i, s = i / (VEC / 4), j = i % (VEC / 4);
      cp_async16(to + (j * slots + s) * 4, param + (c < p.cols ? c : 0), c < p.cols);
    }
  }
}
// The same parameter of vector v straight into registers.
template <int VEC, bool EDGE>
__device__ __forceinline__ void load_param(const float* param, float fill, const Place& p, int v,
                                           F2* out) {
  const int c = v * VEC - p.off;
  if (!EDGE && param != nullptr && v < p.nvec && (reinterpret_cast<uintptr_t>(param) & 15u) == 0) {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(param + c) + j);
      out[2 * j] = f2(q.x, q.y), out[2 * j + 1] = f2(q.z, q.w);
    }
  } else {
    float q[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const bool in = c + j >= 0 && c + j < p.cols;
      q[j] = !in ? 0.0f : (param != nullptr ? __ldg(param + c + j) : fill);
    }
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) out[j] = f2(q[2 * j], q[2 * j + 1]);
  }
}
template <int VEC>
__device__ __forceinline__ void read_param(const float* from, int slots, int s, F2* out) {
#pragma unroll
  for (int j = 0; j < VEC / 4; ++j) {
    const float4 v = reinterpret_cast<const float4*>(from)[j * slots + s];
    out[2 * j] = f2(v.x, v.y), out[2 * j + 1] = f2(v.z, v.w);
  }
}

// Zero the elements of a row's first or last vector that are not its own.
template <int VEC>
__device__ __forceinline__ void mask_vec(F2* a, int e, int cols) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    const bool l = e + 2 * j >= 0 && e + 2 * j < cols, h = e + 2 * j + 1 >= 0 && e + 2 * j + 1 < cols;
    a[j] = f2(l ? f2_lo(a[j]) : 0.0f, h ? f2_hi(a[j]) : 0.0f);
  }
}
// Store a vector's elements that belong to the row, one by one (pieces of 8, 4
// and 2 bytes took longer: more branches).
template <bool BF16, int VEC>
__device__ __forceinline__ void store_part(void* to, int e, int cols, uint4 r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    if (e + j < 0 || e + j >= cols) continue;
    if constexpr (BF16)
      static_cast<uint16_t*>(to)[j] = uint16_t(w[j / 2] >> (16 * (j & 1)));
    else
      static_cast<uint32_t*>(to)[j] = w[j];
  }
}

// Forward. EDGE: rows may start off a 16-byte boundary. MULTI: several warps
// share a row. QUANT also (or only) writes the 1x32 codes and scales of the
// rounded y: a group is 32 / VEC adjacent lanes (cols is a multiple of 32 and
// rows are aligned, so a group never splits over warps).
template <bool BF16, int NV, bool EDGE, bool MULTI, bool QUANT>
__global__ void __launch_bounds__(512)
    k_ln_fwd(const void* __restrict__ x, int64_t rows, int cols, int64_t ldx, int misaligned,
             const float* __restrict__ weight, const float* __restrict__ bias, float eps,
             void* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
             uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, LnSplit split) {
  constexpr int VEC = BF16 ? 8 : 4, NP = VEC / 2, D = ln_depth(NV);
  using V = Vec<BF16, VEC>;
  extern __shared__ __align__(16) uint4 ring[];  // [warps][D][NV][32]
  __shared__ float2 red[2][kLnMaxParts];
  const Place p = place<VEC, NV, EDGE>(split, rows, cols, ldx, misaligned);
  if (MULTI && p.CS > 1) pair_started();
  uint4* const mine = ring + p.warp * (D * NV * 32) + p.lane;

  Walk wx = walk<BF16>(x, rows, ldx, p);
  int to_fetch = p.n;
  int64_t f_row = p.row0;
  const int64_t ends = EDGE ? end_rows<VEC>(ldx) : 1;
  auto fetch = [&](int d) {
    if (to_fetch > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p.v0 + 32 * i < p.nvec) {
          if (EDGE && (f_row < ends || f_row >= rows - ends))
            fetch_vec<BF16, true>(mine + (d * NV + i) * 32, wx.at + 512 * i, wx.first, wx.end);
          else
            fetch_vec<BF16, false>(mine + (d * NV + i) * 32, wx.at + 512 * i, wx.first, wx.end);
        }
    }
    cp_async_commit();
    wx.at += wx.step;
    if (EDGE) f_row += p.stride;
    --to_fetch;
  };
  // vectors past the row's end are zeros that nothing overwrites
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (p.v0 + 32 * i >= p.nvec) {
#pragma unroll
      for (int d = 0; d < D; ++d) mine[(d * NV + i) * 32] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d);
  F2 wk[NV * NP], bk[NV * NP];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<VEC, EDGE>(weight, 1.0f, p, p.v0 + 32 * i, wk + i * NP);
    load_param<VEC, EDGE>(bias, 0.0f, p, p.v0 + 32 * i, bk + i * NP);
  }
  uint8_t* to = static_cast<uint8_t*>(y) +
                (p.row0 * cols + int64_t(p.v0) * VEC - p.off) * (BF16 ? 2 : 4);
  const int64_t to_step = p.stride * cols * (BF16 ? 2 : 4);

  // elements of this warp, and of warp l of the row
  const float inv_n = __fdiv_rn(1.0f, float(cols));
  const int parts = p.W * p.CS, l = p.lane & (p.P - 1);
  const float my_n = part_count<VEC, NV>(p, p.rank * p.W + p.w);
  const float my_inv = my_n > 0.0f ? __fdiv_rn(1.0f, my_n) : 0.0f;
  const float l_n = MULTI && l < parts ? part_count<VEC, NV>(p, l) : 0.0f;
  const float l_inv = l_n > 0.0f ? __fdiv_rn(1.0f, l_n) : 0.0f;
  const float n0 = __shfl_sync(0xFFFFFFFFu, l_n, 0), n1 = __shfl_sync(0xFFFFFFFFu, l_n, 1);
  const float inv0 = __shfl_sync(0xFFFFFFFFu, l_inv, 0);
  const float inv1 = __shfl_sync(0xFFFFFFFFu, l_inv, 1);

  if (MULTI && p.CS > 1) pair_wait_started();
  // the cluster's CTAs walk the same rows; so do the warps of a group
  int d = 0, par = 0;
  int64_t row = p.row0;
  for (int left = p.n; left > 0; --left, row += p.stride, par ^= 1) {
    cp_async_wait<D - 1>();
    F2 a[NV * NP];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      V in;
      in.r = mine[(d * NV + i) * 32];
      in.unpack(a + i * NP);
      if constexpr (EDGE) {
        const int v = p.v0 + 32 * i;
        if (v == 0 || v == p.nvec - 1) mask_vec<VEC>(a + i * NP, v * VEC - p.off, cols);
      }
    }
    fetch(d);
    if (++d == D) d = 0;

    F2 s2 = a[0];
#pragma unroll
    for (int i = 1; i < NV * NP; ++i) s2 = add2(s2, a[i]);
    const float s = warp_sum(__fadd_rn(f2_lo(s2), f2_hi(s2)));
    float mean = __fmul_rn(s, my_inv);
    F2 q2 = f2(0.0f, 0.0f);
    const F2 mm = f2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.v0 + 32 * i;
      if (v >= p.nvec) continue;
      F2 dv[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) dv[j] = add2(a[i * NP + j], mm);
      if constexpr (EDGE) {
        if (v == 0 || v == p.nvec - 1) mask_vec<VEC>(dv, v * VEC - p.off, cols);
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) q2 = fma2(dv[j], dv[j], q2);
    }
    float m2 = warp_sum(__fadd_rn(f2_lo(q2), f2_hi(q2)));
    if constexpr (MULTI) {
      // one barrier a row: the buffer of this parity is written again two
      // rows on, past the next row's barrier
      float2* rd = red[par];
      if (p.CS > 1) {
        if (p.lane < 2) store_pair(&rd[p.rank * p.W + p.w], make_float2(s, m2), p.lane);
        pair_sync();
      } else {
        if (p.lane == 0) rd[p.warp] = make_float2(s, m2);
        group_sync<kLnFwdWarps / 2>(p.g, p.W);
      }
      if (parts == 2) {
        // (every lane the same reads: shorter than shuffles)
        const float2 o0 = rd[p.g * 2], o1 = rd[p.g * 2 + 1];
        mean = __fmul_rn(__fadd_rn(o0.x, o1.x), inv_n);
        const float d0 = __fsub_rn(__fmul_rn(o0.x, inv0), mean);
        const float d1 = __fsub_rn(__fmul_rn(o1.x, inv1), mean);
        m2 = __fadd_rn(__fmaf_rn(__fmul_rn(n0, d0), d0, o0.y),
                       __fmaf_rn(__fmul_rn(n1, d1), d1, o1.y));
      } else {
        const float2 o = l < parts ? rd[p.g * p.W + l] : make_float2(0.0f, 0.0f);
        mean = __fmul_rn(part_sum(o.x, p.P), inv_n);
        const float dm = __fsub_rn(__fmul_rn(o.x, l_inv), mean);
        m2 = part_sum(l < parts ? __fmaf_rn(__fmul_rn(l_n, dm), dm, o.y) : 0.0f, p.P);
      }
    }
    const float rstd = rsqrt_exact(__fmaf_rn(m2, inv_n, eps));
    if (p.v0 == 0) {
      if (mean_out != nullptr) mean_out[row] = mean;
      if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
    // (x - mean) rstd, not x rstd - mean rstd: what is left of x - mean is
    // exact, and a row of one value whose mean has no error gives b
    const F2 nm = f2(-mean, -mean), rs = f2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.v0 + 32 * i;
      const bool in = v < p.nvec;
      if (!QUANT && !in) continue;
      F2 o[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j)
        o[j] = fma2(mul2(add2(a[i * NP + j], nm), rs), wk[i * NP + j], bk[i * NP + j]);
      V out;
      out.pack(o);
      if (in && y != nullptr) {
        if (EDGE && (v == 0 || v == p.nvec - 1))
          store_part<BF16, VEC>(to + 512 * i, v * VEC - p.off, cols, out.r);
        else
          __stcs(reinterpret_cast<uint4*>(to + 512 * i), out.r);
      }
      if constexpr (QUANT) {
        const int64_t at = row * cols + int64_t(v) * VEC;
        if constexpr (BF16) {
          uint32_t am = bf16x8_absmax(out.r);
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          const uint32_t sbyte = scale_byte(am);
          const float mul = inv_scale(sbyte);
          float qv[8];
          F2 r8[4];
          out.unpack(r8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            qv[2 * j] = __fmul_rn(f2_lo(r8[j]), mul);
            qv[2 * j + 1] = __fmul_rn(f2_hi(r8[j]), mul);
          }
          const uint32_t word = sbyte == 0xFFu ? 0u : e2m1x8_rn(qv);
          if (in) {
            *reinterpret_cast<uint32_t*>(codes + at / 2) = word;
            if ((p.lane & 3) == 0) scales[at / 32] = static_cast<uint8_t>(sbyte);
          }
        } else {
          uint32_t am = max(max(out.r.x & 0x7FFFFFFFu, out.r.y & 0x7FFFFFFFu),
                            max(out.r.z & 0x7FFFFFFFu, out.r.w & 0x7FFFFFFFu));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 4));
          const uint32_t sbyte = scale_byte(am);
          const float mul = inv_scale(sbyte);
          const float qv[8] = {__fmul_rn(__uint_as_float(out.r.x), mul),
                               __fmul_rn(__uint_as_float(out.r.y), mul),
                               __fmul_rn(__uint_as_float(out.r.z), mul),
                               __fmul_rn(__uint_as_float(out.r.w), mul), 0, 0, 0, 0};
          const uint32_t word = sbyte == 0xFFu ? 0u : e2m1x8_rn(qv);
          if (in) {
            *reinterpret_cast<uint16_t*>(codes + at / 2) = static_cast<uint16_t>(word);
            if ((p.lane & 7) == 0) scales[at / 32] = static_cast<uint8_t>(sbyte);
          }
        }
      }
    }
    to += to_step;
  }
  cp_async_wait<0>();
  if (p.CS > 1) pair_sync();  // no CTA ends while the other may still write to it
}

// Rows wider than the registers of a cluster: one CTA a row, three passes
// over it (the second and third from L2).
__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < kLnGenThreads / 32; ++i) t = __fadd_rn(t, sh[i]);
  return t;
}
template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t e) {
  return BF16 ? __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + e)) << 16)
              : __ldg(static_cast<const float*>(p) + e);
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t e, float v) {
  if (BF16)
    static_cast<uint16_t*>(p)[e] = uint16_t(pack_bf16x2(v, 0.0f));
  else
    static_cast<float*>(p)[e] = v;
}

template <bool BF16>
__global__ void __launch_bounds__(kLnGenThreads)
    k_ln_fwd_wide(const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx,
                  const float* __restrict__ weight, const float* __restrict__ bias, float eps,
                  void* __restrict__ y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out, uint8_t* __restrict__ codes,
                  uint8_t* __restrict__ scales) {
  __shared__ float sh[kLnGenThreads / 32];
  const float n = float(cols);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t x0 = row * ldx, y0 = row * cols;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kLnGenThreads)
      s = __fadd_rn(s, load1<BF16>(x, x0 + c));
    const float mean = __fdiv_rn(block_sum(s, sh), n);
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kLnGenThreads) {
      const float d = __fsub_rn(load1<BF16>(x, x0 + c), mean);
      q = __fmaf_rn(d, d, q);
    }
    const float rstd = rsqrt_exact(__fadd_rn(__fdiv_rn(block_sum(q, sh), n), eps));
    if (threadIdx.x == 0) {
      if (mean_out != nullptr) mean_out[row] = mean;
      if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
    // whole groups of 32 columns per warp, so that a group can be quantized
    for (int64_t c0 = (threadIdx.x & ~31u); c0 < cols; c0 += kLnGenThreads) {
      const int lane = threadIdx.x & 31;
      const int64_t c = c0 + lane;
      float v = 0.0f;
      if (c < cols) {
        const float h = __fmul_rn(__fsub_rn(load1<BF16>(x, x0 + c), mean), rstd);
        v = __fmaf_rn(h, weight != nullptr ? __ldg(weight + c) : 1.0f,
                      bias != nullptr ? __ldg(bias + c) : 0.0f);
        if (BF16) v = __uint_as_float(pack_bf16x2(v, 0.0f) << 16);
        if (y != nullptr) store1<BF16>(y, y0 + c, v);
      }
      if (codes != nullptr) {
        uint32_t am = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        const uint32_t sb = scale_byte(am);
        const float mine = __fmul_rn(v, inv_scale(sb));
        float qv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) qv[j] = __shfl_sync(0xFFFFFFFFu, mine, (lane & ~7) + j);
        const uint32_t word = sb == 0xFFu ? 0u : e2m1x8_rn(qv);
        if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(codes + (y0 + c) / 2) = word;
        if (lane == 0) scales[(y0 + c) / 32] = static_cast<uint8_t>(sb);
      }
    }
  }
}

// Backward; PARAMS = false leaves dw and db out.
template <bool BF16, int NV, bool EDGE, bool MULTI, bool PARAMS>
__global__ void __launch_bounds__(512)
    k_ln_bwd(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows, int cols,
             int64_t lddy, int64_t ldx, int misaligned, const float* __restrict__ weight,
             const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
             void* __restrict__ dx, float* __restrict__ partial, LnSplit split) {
  constexpr int VEC = BF16 ? 8 : 4, NP = VEC / 2, D = ln_depth(NV);
  constexpr bool kW = NV == 1;
  using V = Vec<BF16, VEC>;
  extern __shared__ __align__(16) uint4 ring[];  // [warps][D][2 NV][32], then w
  __shared__ float2 red[2][kLnMaxParts];
  const Place p = place<VEC, NV, EDGE>(split, rows, cols, ldx, misaligned);
  if (MULTI && p.CS > 1) pair_started();
  const int slots = p.W * NV * 32, s0 = p.w * NV * 32 + p.lane;
  float* const sw = reinterpret_cast<float*>(ring + (blockDim.x >> 5) * (D * 2 * NV * 32));
  uint4* const mine = ring + p.warp * (D * 2 * NV * 32) + p.lane;

  Walk wx = walk<BF16>(x, rows, ldx, p), wg = walk<BF16>(dy, rows, lddy, p);
  int to_fetch = p.n;
  int64_t f_row = p.row0;
  const int64_t ends = EDGE ? end_rows<VEC>(ldx < lddy ? ldx : lddy) : 1;
  auto fetch = [&](int d) {
    if (to_fetch > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p.v0 + 32 * i < p.nvec) {
          uint4* const to = mine + (d * NV + i) * 64;
          if (EDGE && (f_row < ends || f_row >= rows - ends)) {
            fetch_vec<BF16, true>(to, wx.at + 512 * i, wx.first, wx.end);
            fetch_vec<BF16, true>(to + 32, wg.at + 512 * i, wg.first, wg.end);
          } else {
            fetch_vec<BF16, false>(to, wx.at + 512 * i, wx.first, wx.end);
            fetch_vec<BF16, false>(to + 32, wg.at + 512 * i, wg.first, wg.end);
          }
        }
    }
    cp_async_commit();
    wx.at += wx.step, wg.at += wg.step;
    if (EDGE) f_row += p.stride;
    --to_fetch;
  };
  // vectors past the row's end are zeros that nothing overwrites
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (p.v0 + 32 * i >= p.nvec) {
#pragma unroll
      for (int d = 0; d < D; ++d)
        mine[(d * NV + i) * 64] = mine[(d * NV + i) * 64 + 32] = make_uint4(0, 0, 0, 0);
    }
  if constexpr (!kW) stage_param<VEC, NV, EDGE>(weight, 1.0f, p, sw);
  cp_async_commit();
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d);
  F2 wk[kW ? NP : 1];
  if constexpr (kW) load_param<VEC, EDGE>(weight, 1.0f, p, p.v0, wk);
  uint8_t* to = static_cast<uint8_t*>(dx) +
                (p.row0 * cols + int64_t(p.v0) * VEC - p.off) * (BF16 ? 2 : 4);
  const int64_t to_step = p.stride * cols * (BF16 ? 2 : 4);

  const float inv_n = __fdiv_rn(1.0f, float(cols));
  const int parts = p.W * p.CS, l = p.lane & (p.P - 1);
  const F2 zero = f2(0.0f, 0.0f);
  F2 aw[PARAMS ? NV * NP : 1], ab[PARAMS ? NV * NP : 1];
  if constexpr (PARAMS) {
#pragma unroll
    for (int k = 0; k < NV * NP; ++k) aw[k] = ab[k] = zero;
  }
  float nmean = 0.0f, nrstd = 0.0f;
  const float *mp = mean_in + p.row0, *rp = rstd_in + p.row0;
  if (p.n > 0) nmean = __ldg(mp), nrstd = __ldg(rp);
  if constexpr (!kW) {
    cp_async_wait<D>();  // the weight
    __syncthreads();
  }
  if (MULTI && p.CS > 1) pair_wait_started();

  int d = 0, par = 0;
  for (int left = p.n; left > 0; --left, par ^= 1) {
    const float mean = nmean, rstd = nrstd;
    mp += p.stride, rp += p.stride;
    if (left > 1) nmean = __ldg(mp), nrstd = __ldg(rp);
    cp_async_wait<D - 1>();
    F2 h[NV * NP], g[NV * NP];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      V in;
      in.r = mine[(d * NV + i) * 64];
      in.unpack(h + i * NP);
      in.r = mine[(d * NV + i) * 64 + 32];
      in.unpack(g + i * NP);
      if constexpr (EDGE) {
        const int v = p.v0 + 32 * i;
        if (v == 0 || v == p.nvec - 1) {
          mask_vec<VEC>(h + i * NP, v * VEC - p.off, cols);
          mask_vec<VEC>(g + i * NP, v * VEC - p.off, cols);
        }
      }
    }
    fetch(d);
    if (++d == D) d = 0;

    // (an element outside the row has g = 0: it adds nothing anywhere)
    const F2 nm = f2(-mean, -mean), rs = f2(rstd, rstd);
    F2 c1 = zero, c2 = zero;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      F2 wv[NP];
      if constexpr (!kW) read_param<VEC>(sw, slots, s0 + 32 * i, wv);
      if constexpr (kW)
#pragma unroll
        for (int j = 0; j < NP; ++j) wv[j] = wk[j];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int k = i * NP + j;
        h[k] = mul2(add2(h[k], nm), rs);
        if constexpr (PARAMS) {
          aw[k] = fma2(g[k], h[k], aw[k]);
          ab[k] = add2(ab[k], g[k]);
        }
        g[k] = mul2(g[k], wv[j]);
        c1 = add2(c1, g[k]);
        c2 = fma2(g[k], h[k], c2);
      }
    }
    const float half_sum = warp_sum2(__fadd_rn(f2_lo(c1), f2_hi(c1)),
                                     __fadd_rn(f2_lo(c2), f2_hi(c2)), p.lane);
    float s1, s2;
    if constexpr (MULTI) {
      float2* rd = red[par];
      if (p.CS > 1) {
        const float other = __shfl_sync(0xFFFFFFFFu, half_sum, 16);
        const float mine_ = __shfl_sync(0xFFFFFFFFu, half_sum, 0);
        if (p.lane < 2) store_pair(&rd[p.rank * p.W + p.w], make_float2(mine_, other), p.lane);
        pair_sync();
      } else {
        if ((p.lane & 15) == 0)
          reinterpret_cast<float*>(&rd[p.warp])[p.lane >> 4] = half_sum;
        group_sync<kLnBwdWarps / 2>(p.g, p.W);
      }
      if (parts <= 4) {
        // (every lane the same reads: shorter than shuffles)
        s1 = s2 = 0.0f;
        for (int k = 0; k < parts; ++k) {
          const float2 o = rd[p.g * p.W + k];
          s1 = __fadd_rn(s1, o.x), s2 = __fadd_rn(s2, o.y);
        }
      } else {
        const float2 o = l < parts ? rd[p.g * p.W + l] : make_float2(0.0f, 0.0f);
        s1 = part_sum(o.x, p.P);
        s2 = part_sum(o.y, p.P);
      }
    } else {
      s1 = __shfl_sync(0xFFFFFFFFu, half_sum, 0);
      s2 = __shfl_sync(0xFFFFFFFFu, half_sum, 16);
    }
    // dx = g rstd - (c1 + h c2) rstd / n
    const float ri = -__fmul_rn(rstd, inv_n), m1 = __fmul_rn(s1, ri), m2 = __fmul_rn(s2, ri);
    const F2 k1 = f2(m1, m1), k2 = f2(m2, m2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.v0 + 32 * i;
      if (v >= p.nvec) continue;
      F2 o[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int k = i * NP + j;
        o[j] = fma2(h[k], k2, fma2(g[k], rs, k1));
      }
      V out;
      out.pack(o);
      if (EDGE && (v == 0 || v == p.nvec - 1))
        store_part<BF16, VEC>(to + 512 * i, v * VEC - p.off, cols, out.r);
      else
        __stcs(reinterpret_cast<uint4*>(to + 512 * i), out.r);
    }
    to += to_step;
  }
  cp_async_wait<0>();

  if constexpr (PARAMS) {
    // the groups of a CTA (same columns, same `off`) add into shared memory
    // one after the other; the last one writes the partial row (a CTA whose
    // first group has no row has none: the workspace ends before its place)
    const bool used = p.row0 - p.g * (EDGE ? VEC : 1) < rows;
    float* pw = partial + int64_t(blockIdx.x / p.CS) * 2 * cols;
    float* sacc = reinterpret_cast<float*>(ring);  // [2][slots VEC]
    const int G = (blockDim.x >> 5) / p.W;
    if (G > 1) __syncthreads();  // every group is done with the ring
    for (int g = 0; g < G; ++g) {
      if (p.g == g) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c0 = (p.v0 + 32 * i) * VEC - p.off;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int k = i * NP + j / 2, at = j * slots + s0 + 32 * i;
            float a = (j & 1) ? f2_hi(aw[k]) : f2_lo(aw[k]);
            float b = (j & 1) ? f2_hi(ab[k]) : f2_lo(ab[k]);
            if (g > 0) a = __fadd_rn(a, sacc[at]), b = __fadd_rn(b, sacc[slots * VEC + at]);
            if (g + 1 < G) {
              sacc[at] = a, sacc[slots * VEC + at] = b;
            } else if (used && c0 + j >= 0 && c0 + j < cols) {
              pw[c0 + j] = a, pw[cols + c0 + j] = b;
            }
          }
        }
      }
      if (G > 1) __syncthreads();
    }
  }
  if (p.CS > 1) pair_sync();
}

// Backward, aligned rows of at most kLnRowWarps warps with one vector a thread:
// R rows of the group at a time. The sums of R rows are reduced together (2 R values
// over 32 lanes by exchanging halves: R = 4 takes 9 shuffles and one barrier
// instead of 40 and 4), and x and dy are read from shared memory a second time
// for dx and the column sums, so that a thread holds little: more warps run,
// and the R rows are independent work. 12608 x 1536 bf16: 27.6 us, a row at a
// time (k_ln_bwd) 31.5 us; 12608 x 384: 13.5 and 19.1 us.
template <int N>
__device__ __forceinline__ float exchange_sum(float (&v)[N], int lane, int mask) {
  if constexpr (N == 1) {
    float t = v[0];
    for (int o = mask; o > 0; o >>= 1) t = __fadd_rn(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
    return t;
  } else {
    const bool up = (lane & mask) != 0;
    float h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float give = up ? v[i] : v[i + N / 2], keep = up ? v[i + N / 2] : v[i];
      h[i] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, mask));
    }
    return exchange_sum<N / 2>(h, lane, mask / 2);
  }
}

template <bool BF16, bool MULTI, bool PARAMS>
__global__ void __launch_bounds__(kLnRowWarps * 32)
    k_ln_bwd_rows(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows, int cols,
                  int64_t lddy, int64_t ldx, const float* __restrict__ weight,
                  const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                  void* __restrict__ dx, float* __restrict__ partial, LnSplit split) {
  constexpr int VEC = BF16 ? 8 : 4, NP = VEC / 2, R = 4, NV = 2 * R;  // NV sums
  constexpr int kPer = 32 / NV;  // lanes that hold the same sum
  using V = Vec<BF16, VEC>;
  extern __shared__ __align__(16) uint4 ring[];  // [warps][2][R][2][32]
  __shared__ float red[2][kLnRowWarps][NV];
  const Place p = place<VEC, 1, false>(split, rows, cols, ldx, 0);
  uint4* const mine = ring + p.warp * (2 * R * 64) + p.lane;
  const bool live = p.v0 < p.nvec;
  const int e = p.v0 * VEC;

  Walk wx = walk<BF16>(x, rows, ldx, p), wg = walk<BF16>(dy, rows, lddy, p);
  int to_fetch = p.n;
  const float *mp = mean_in + p.row0, *rp = rstd_in + p.row0;
  float nmean[R], nrstd[R];
  auto fetch = [&](int b) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (to_fetch > 0) {
        uint4* const to = mine + (b * R + r) * 64;
        if (live) {
          fetch_vec<BF16, false>(to, wx.at, wx.first, wx.end);
          fetch_vec<BF16, false>(to + 32, wg.at, wg.first, wg.end);
        }
      }
      wx.at += wx.step, wg.at += wg.step;
      --to_fetch;
    }
    cp_async_commit();
  };
  auto fetch_stats = [&](int left) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      nmean[r] = r < left ? __ldg(mp) : 0.0f;
      nrstd[r] = r < left ? __ldg(rp) : 0.0f;
      mp += p.stride, rp += p.stride;
    }
  };
  if (!live) {
#pragma unroll
    for (int i = 0; i < 2 * R * 2; ++i) mine[i * 32] = make_uint4(0, 0, 0, 0);
  }
  fetch(0);
  fetch(1);
  fetch_stats(p.n);
  F2 wk[NP];
  load_param<VEC, false>(weight, 1.0f, p, p.v0, wk);
  uint8_t* to = static_cast<uint8_t*>(dx) + (p.row0 * cols + e) * (BF16 ? 2 : 4);
  const int64_t to_step = p.stride * cols * (BF16 ? 2 : 4);
  const float inv_n = __fdiv_rn(1.0f, float(cols));
  const F2 zero = f2(0.0f, 0.0f);
  F2 aw[PARAMS ? NP : 1], ab[PARAMS ? NP : 1];
  if constexpr (PARAMS) {
#pragma unroll
    for (int k = 0; k < NP; ++k) aw[k] = ab[k] = zero;
  }

  // h = (x - mean) rstd and dy of row r of buffer b
  auto read = [&](int b, int r, float mean, float rstd, F2* h, F2* g) {
    V in;
    in.r = mine[(b * R + r) * 64];
    in.unpack(h);
    in.r = mine[(b * R + r) * 64 + 32];
    in.unpack(g);
    const F2 nm = f2(-mean, -mean), rs = f2(rstd, rstd);
#pragma unroll
    for (int k = 0; k < NP; ++k) h[k] = mul2(add2(h[k], nm), rs);
  };

  int b = 0;
  for (int left = p.n; left > 0; left -= R, b ^= 1) {
    float mean[R], rstd[R], s[NV];
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = nmean[r], rstd[r] = nrstd[r];
    fetch_stats(left - R);
    cp_async_wait<1>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 h[NP], g[NP], c1 = zero, c2 = zero;
      if (r < left) {
        read(b, r, mean[r], rstd[r], h, g);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const F2 gw = mul2(g[k], wk[k]);
          c1 = add2(c1, gw);
          c2 = fma2(gw, h[k], c2);
        }
      }
      s[2 * r] = __fadd_rn(f2_lo(c1), f2_hi(c1));
      s[2 * r + 1] = __fadd_rn(f2_lo(c2), f2_hi(c2));
    }
    // lane l then holds the warp's sum l / kPer
    float sum = exchange_sum<NV>(s, p.lane, 16);
    if constexpr (MULTI) {
      // one barrier for R rows: the buffer of this parity is written again two
      // rounds on, past the next round's barrier
      if (p.lane % kPer == 0) red[b][p.warp][p.lane / kPer] = sum;
      group_sync<kLnRowGroups>(p.g, p.W);
      sum = 0.0f;
      for (int k = 0; k < p.W; ++k)
        sum = __fadd_rn(sum, red[b][p.g * p.W + k][p.lane / kPer]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float s1 = __shfl_sync(0xFFFFFFFFu, sum, 2 * r * kPer);
      const float s2 = __shfl_sync(0xFFFFFFFFu, sum, (2 * r + 1) * kPer);
      if (r < left) {
        F2 h[NP], g[NP], o[NP];
        read(b, r, mean[r], rstd[r], h, g);
        // dx = g rstd - (c1 + h c2) rstd / n
        const float ri = -__fmul_rn(rstd[r], inv_n);
        const float m1 = __fmul_rn(s1, ri), m2 = __fmul_rn(s2, ri);
        const F2 k1 = f2(m1, m1), k2 = f2(m2, m2), rs = f2(rstd[r], rstd[r]);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          if constexpr (PARAMS) {
            aw[k] = fma2(g[k], h[k], aw[k]);
            ab[k] = add2(ab[k], g[k]);
          }
          o[k] = fma2(h[k], k2, fma2(mul2(g[k], wk[k]), rs, k1));
        }
        V out;
        out.pack(o);
        if (live) __stcs(reinterpret_cast<uint4*>(to), out.r);
      }
      to += to_step;
    }
    fetch(b);
  }
  cp_async_wait<0>();

  if constexpr (PARAMS) {
    // the groups of a CTA (same columns) add into shared memory
    // one after the other; the last one writes the partial row
    float* pw = partial + int64_t(blockIdx.x) * 2 * cols;
    float* sacc = reinterpret_cast<float*>(ring);  // [2][VEC][slots]
    const int G = (blockDim.x >> 5) / p.W, slots = p.W * 32;
    if (G > 1) __syncthreads();  // every group is done with the ring
    for (int gi = 0; gi < G; ++gi) {
      if (p.g == gi) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int at = j * slots + p.v0;
          float a = (j & 1) ? f2_hi(aw[j / 2]) : f2_lo(aw[j / 2]);
          float bb = (j & 1) ? f2_hi(ab[j / 2]) : f2_lo(ab[j / 2]);
          if (gi > 0) a = __fadd_rn(a, sacc[at]), bb = __fadd_rn(bb, sacc[slots * VEC + at]);
          if (gi + 1 < G) {
            sacc[at] = a, sacc[slots * VEC + at] = bb;
          } else if (e + j < cols) {
            pw[e + j] = a, pw[cols + e + j] = bb;
          }
        }
      }
      if (G > 1) __syncthreads();
    }
  }
}

// Rows wider than the registers of a cluster: dx with one CTA a row, and the
// column sums by a kernel of their own that reads x and dy again.
template <bool BF16>
__global__ void __launch_bounds__(kLnGenThreads)
    k_ln_bwd_wide(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows,
                  int64_t cols, int64_t lddy, int64_t ldx, const float* __restrict__ weight,
                  const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                  void* __restrict__ dx) {
  __shared__ float sh[kLnGenThreads / 32];
  const float n = float(cols);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float mean = mean_in[row], rstd = rstd_in[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kLnGenThreads) {
      const float h = __fmul_rn(__fsub_rn(load1<BF16>(x, row * ldx + c), mean), rstd);
      const float g = __fmul_rn(load1<BF16>(dy, row * lddy + c),
                                weight != nullptr ? __ldg(weight + c) : 1.0f);
      c1 = __fadd_rn(c1, g);
      c2 = __fmaf_rn(g, h, c2);
    }
    c1 = __fdiv_rn(block_sum(c1, sh), n);
    c2 = __fdiv_rn(block_sum(c2, sh), n);
    for (int64_t c = threadIdx.x; c < cols; c += kLnGenThreads) {
      const float h = __fmul_rn(__fsub_rn(load1<BF16>(x, row * ldx + c), mean), rstd);
      const float g = __fmul_rn(load1<BF16>(dy, row * lddy + c),
                                weight != nullptr ? __ldg(weight + c) : 1.0f);
      store1<BF16>(dx, row * cols + c,
                   __fmul_rn(__fsub_rn(__fmaf_rn(-h, c2, g), c1), rstd));
    }
  }
}
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_ln_bwd_wide_params(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows,
                         int64_t cols, int64_t lddy, int64_t ldx,
                         const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                         float* __restrict__ partial) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= cols) return;
  float a = 0.0f, b = 0.0f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float h =
        __fmul_rn(__fsub_rn(load1<BF16>(x, row * ldx + c), mean_in[row]), rstd_in[row]);
    const float g = load1<BF16>(dy, row * lddy + c);
    a = __fmaf_rn(g, h, a);
    b = __fadd_rn(b, g);
  }
  float* pw = partial + int64_t(blockIdx.y) * 2 * cols;
  pw[c] = a, pw[cols + c] = b;
}

// dw and db from the `n` partial rows [2][cols]: a CTA takes 32 of the 2 cols
// columns, warp w adds rows w, w + 32, ..., and the 32 warps' sums are added
// in order.
__global__ void __launch_bounds__(kLnRedThreads)
    k_ln_params(const float* __restrict__ partial, int n, int64_t cols, float* __restrict__ dw,
                float* __restrict__ db) {
  __shared__ float sh[kLnRedThreads / 32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < 2 * cols) {
    int r = w;
    for (; r + 96 < n; r += 128) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = __ldcg(partial + int64_t(r + 32 * u) * 2 * cols + c);
#pragma unroll
      for (int u = 0; u < 4; ++u) s = __fadd_rn(s, v[u]);
    }
    for (; r < n; r += 32) s = __fadd_rn(s, __ldcg(partial + int64_t(r) * 2 * cols + c));
  }
  sh[w][lane] = s;
  __syncthreads();
  s = warp_sum(sh[lane][w]);  // warp w: column w of the 32
  const int64_t cw = int64_t(blockIdx.x) * 32 + w;
  if (lane == 0 && cw < 2 * cols) (cw < cols ? dw[cw] : db[cw - cols]) = s;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

struct LnShape {
  int nv, threads;
  LnSplit split;
};

int sm_count() {
  static thread_local int known_dev = -1, known = 148;
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev != known_dev) {
    cudaDeviceGetAttribute(&known, cudaDevAttrMultiProcessorCount, dev);
    known_dev = dev;
  }
  return known;
}

// Vectors per thread and warps per row: `big` vectors (whose parameters still
// fit in registers), one where a warp then holds a row, or where rows are few
// (less than two an SM: one vector a thread spreads a row over the most
// threads). Rows that 16 warps cannot hold take a cluster of two CTAs. Rows
// that need less than a CTA of `block_warps` warps share one.
// 12608 x 1536 bf16, forward: 24 elements a thread 14.8 us, 48 (one warp a
// row, parameters in shared memory, whose bandwidth then binds) 20.2 us.
bool ln_shape(int64_t nvec, int big, int64_t rows, int block_warps, LnShape* s) {
  const bool few = rows < 2 * int64_t(sm_count());
  s->nv = nvec <= 32 || (few && nvec <= 32 * kLnMaxWarps) ? 1 : big;
  int64_t W = (nvec + 32 * s->nv - 1) / (32 * s->nv);
  s->split.CS = 1;
  if (W > kLnMaxWarps) {
    s->split.CS = 2;
    W = (W + 1) / 2;
    if (W > kLnMaxWarps) return false;
  }
  s->split.W = int(W);
  s->split.P = 1;
  while (s->split.P < s->split.W * s->split.CS) s->split.P *= 2;
  s->split.G = few || s->split.CS > 1 || W >= block_warps ? 1 : int(block_warps / W);
  s->threads = 32 * s->split.W * s->split.G;
  return true;
}

// Whether rows of these tensors (base, stride) can move as 16-byte vectors:
// every row on a boundary (*edge = false), or all of them without padding
// and equally far off it (*edge = true, *misaligned = elements).
bool vector_rows(const void* const* p, const int64_t* ld, int n, int64_t cols, int size,
                 bool* edge, int* misaligned) {
  const int vec = 16 / size;
  bool whole = cols % vec == 0, dense = true;
  for (int i = 0; i < n; ++i) {
    if (p[i] == nullptr) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p[i]) & 15u;
    if (a != 0 || (ld[i] * size) % 16 != 0) whole = false;
    if (ld[i] != cols || a != (reinterpret_cast<uintptr_t>(p[0]) & 15u)) dense = false;
  }
  *edge = !whole;
  *misaligned = int((reinterpret_cast<uintptr_t>(p[0]) & 15u) / size);
  return whole || dense;
}

// Persistent grid of whole clusters; with rows off the boundary a multiple of
// the vector length of them (see Place).
int ln_grid(const void* kern, const LnShape& sh, size_t smem, int64_t rows, bool edge, int vec,
            int64_t most) {
  const int64_t unit = edge ? vec : 1;
  int64_t want = ((rows + unit - 1) / unit + sh.split.G - 1) / sh.split.G * unit;
  if (want > most) want = most;
  const int64_t n =
      persistent_grid(kern, sh.threads, smem, want * sh.split.CS) / sh.split.CS / unit * unit;
  return int((n < unit ? unit : n) * sh.split.CS);
}

// How many of a backward grid's `blocks` clusters have rows, the first ones
// (see Place): each writes a partial row of dw and db. At most `rows`, also
// where the grid was rounded up to the vector length.
int64_t ln_partials(const LnShape& sh, int64_t rows, bool edge, int vec, int64_t blocks) {
  const int64_t unit = edge ? vec : 1, round = sh.split.G * unit;
  const int64_t rest = rows % round < unit ? rows % round : unit;
  const int64_t n = rows / round * unit + rest;
  return n < blocks ? n : blocks;
}

template <typename... P, typename... A>
cudaError_t ln_launch(void (*kern)(P...), int grid, const LnShape& sh, size_t smem,
                      cudaStream_t s, A... args) {
  if (sh.split.CS == 1) {
    kern<<<unsigned(grid), unsigned(sh.threads), smem, s>>>(args...);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(sh.threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(sh.split.CS);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct FwdArgs {
  const void* x;
  int64_t rows, cols, ldx;
  const float *weight, *bias;
  float eps;
  void* y;
  float *mean, *rstd;
  uint8_t *codes, *scales;
  cudaStream_t s;
};

template <bool BF16, int NV, bool EDGE, bool MULTI, bool QUANT>
cudaError_t fwd_launch(const FwdArgs& a, const LnShape& sh, int misaligned) {
  constexpr int VEC = BF16 ? 8 : 4;
  auto kern = k_ln_fwd<BF16, NV, EDGE, MULTI, QUANT>;
  const void* k = reinterpret_cast<const void*>(kern);
  const size_t smem = size_t(sh.threads) * NV * 16 * ln_depth(NV);
  const cudaError_t e = allow_smem(k, smem);
  if (e != cudaSuccess) return e;
  const int grid = ln_grid(k, sh, smem, a.rows, EDGE, VEC, int64_t(1) << 30);
  return ln_launch(kern, grid, sh, smem, a.s, a.x, a.rows, int(a.cols), a.ldx, misaligned,
                   a.weight, a.bias, a.eps, a.y, a.mean, a.rstd, a.codes, a.scales, sh.split);
}

template <bool BF16, int NV, bool MULTI>
cudaError_t fwd_nv(const FwdArgs& a, const LnShape& sh, bool edge, int misaligned) {
  if (a.codes != nullptr) return fwd_launch<BF16, NV, false, MULTI, true>(a, sh, 0);
  return edge ? fwd_launch<BF16, NV, true, MULTI, false>(a, sh, misaligned)
              : fwd_launch<BF16, NV, false, MULTI, false>(a, sh, 0);
}

template <bool BF16>
cudaError_t fwd_any(const FwdArgs& a) {
  constexpr int kSize = BF16 ? 2 : 4, VEC = 16 / kSize;
  // Vectors a thread, more (32 elements, the parameters in registers beside
  // them at 128 registers a thread) where fewer lanes are then idle, or where
  // a row needs a cluster otherwise (whose barrier a row cost more than a few
  // spilled registers). bf16, 3 / 4: 8192 x 4096 32.3 / 25.3 us, 4096 x 14336
  // 103 / 49 us; fp32, 4 / 8: 4096 x 8192 45.4 / 47.5 us, 4096 x 14336
  // 143 / 86 us.
  constexpr int kBig = BF16 ? 3 : 4, kWide = BF16 ? 4 : 8;
  LnShape sh;
  bool edge = false;
  int mis = 0;
  const void* const ptrs[] = {a.x, a.y};
  const int64_t lds[] = {a.ldx, a.cols};
  const bool vec = a.cols <= kLnMaxCols && vector_rows(ptrs, lds, 2, a.cols, kSize, &edge, &mis);
  const int64_t nvec = (a.cols + VEC - 1) / VEC + (edge ? 1 : 0);
  const int64_t wb = (nvec + 32 * kBig - 1) / (32 * kBig);
  const int64_t ww = (nvec + 32 * kWide - 1) / (32 * kWide);
  const bool more = wb > kLnMaxWarps || ww * kWide < wb * kBig;
  if (vec &&
      !(edge && a.codes != nullptr) &&
      ln_shape(nvec, more ? kWide : kBig, a.rows, kLnFwdWarps, &sh)) {
    const bool multi = sh.split.W * sh.split.CS > 1;
    if (sh.nv == 1)
      return multi ? fwd_nv<BF16, 1, true>(a, sh, edge, mis)
                   : fwd_nv<BF16, 1, false>(a, sh, edge, mis);
    if (more) {
      if constexpr (BF16)
        if (!multi) return fwd_nv<BF16, kWide, false>(a, sh, edge, mis);
      return fwd_nv<BF16, kWide, true>(a, sh, edge, mis);
    }
    return multi ? fwd_nv<BF16, kBig, true>(a, sh, edge, mis)
                 : fwd_nv<BF16, kBig, false>(a, sh, edge, mis);
  }
  auto kern = k_ln_fwd_wide<BF16>;
  const int grid =
      persistent_grid(reinterpret_cast<const void*>(kern), kLnGenThreads, 0, a.rows);
  kern<<<grid, kLnGenThreads, 0, a.s>>>(a.x, a.rows, a.cols, a.ldx, a.weight, a.bias, a.eps, a.y,
                                        a.mean, a.rstd, a.codes, a.scales);
  return cudaGetLastError();
}

struct BwdArgs {
  const void *dy, *x;
  int64_t rows, cols, lddy, ldx;
  const float *weight, *mean, *rstd;
  void* dx;
  float *dw, *db, *partial;
  cudaStream_t s;
};

cudaError_t params_launch(const BwdArgs& a, int n) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((2 * a.cols + 31) / 32));
  cfg.blockDim = dim3(kLnRedThreads);
  cfg.stream = a.s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ln_params, static_cast<const float*>(a.partial), n, a.cols,
                            a.dw, a.db);
}

template <bool BF16, int NV, bool EDGE, bool MULTI, bool PARAMS>
cudaError_t bwd_launch(const BwdArgs& a, const LnShape& sh, int misaligned) {
  constexpr int VEC = BF16 ? 8 : 4;
  auto kern = k_ln_bwd<BF16, NV, EDGE, MULTI, PARAMS>;
  const void* k = reinterpret_cast<const void*>(kern);
  const size_t params = size_t(sh.split.W) * NV * 32 * VEC * 4;
  size_t smem = size_t(sh.threads) * 2 * NV * 16 * ln_depth(NV) + params;
  if (smem < 2 * params) smem = 2 * params;  // the groups' sums, at the end
  cudaError_t e = allow_smem(k, smem);
  if (e != cudaSuccess) return e;
  const int grid = ln_grid(k, sh, smem, a.rows, EDGE, VEC, kLnMaxPartials);
  e = ln_launch(kern, grid, sh, smem, a.s, a.dy, a.x, a.rows, int(a.cols), a.lddy, a.ldx,
                misaligned, a.weight, a.mean, a.rstd, a.dx, a.partial, sh.split);
  if (e != cudaSuccess || !PARAMS) return e;
  return params_launch(a, int(ln_partials(sh, a.rows, EDGE, VEC, grid / sh.split.CS)));
}

template <bool BF16, bool MULTI, bool PARAMS>
cudaError_t bwd_rows(const BwdArgs& a, const LnShape& sh) {
  constexpr int VEC = BF16 ? 8 : 4;
  auto kern = k_ln_bwd_rows<BF16, MULTI, PARAMS>;
  const void* k = reinterpret_cast<const void*>(kern);
  const size_t smem = size_t(sh.threads) * 2 * 4 * 2 * 16;
  cudaError_t e = allow_smem(k, smem);
  if (e != cudaSuccess) return e;
  const int grid = ln_grid(k, sh, smem, a.rows, false, VEC, kLnMaxPartials);
  e = ln_launch(kern, grid, sh, smem, a.s, a.dy, a.x, a.rows, int(a.cols), a.lddy, a.ldx,
                a.weight, a.mean, a.rstd, a.dx, a.partial, sh.split);
  if (e != cudaSuccess || !PARAMS) return e;
  return params_launch(a, int(ln_partials(sh, a.rows, false, VEC, grid)));
}
template <bool BF16>
cudaError_t bwd_rows_any(const BwdArgs& a, int64_t nvec) {
  LnShape sh;
  const int W = int((nvec + 31) / 32);
  sh.nv = 1;
  sh.split.W = W, sh.split.CS = 1, sh.split.P = 1;
  // groups share a CTA (at most kLnRowGroups, whose barriers are numbered)
  const int G = W >= kLnRowShare ? 1 : kLnRowShare / W;
  sh.split.G = W > 1 && G > kLnRowGroups ? kLnRowGroups : G;
  sh.threads = 32 * W * sh.split.G;
  if (W > 1)
    return a.dw != nullptr ? bwd_rows<BF16, true, true>(a, sh)
                           : bwd_rows<BF16, true, false>(a, sh);
  return a.dw != nullptr ? bwd_rows<BF16, false, true>(a, sh)
                         : bwd_rows<BF16, false, false>(a, sh);
}

template <bool BF16, int NV, bool MULTI>
cudaError_t bwd_nv(const BwdArgs& a, const LnShape& sh, bool edge, int misaligned) {
  if (a.dw != nullptr)
    return edge ? bwd_launch<BF16, NV, true, MULTI, true>(a, sh, misaligned)
                : bwd_launch<BF16, NV, false, MULTI, true>(a, sh, 0);
  return edge ? bwd_launch<BF16, NV, true, MULTI, false>(a, sh, misaligned)
              : bwd_launch<BF16, NV, false, MULTI, false>(a, sh, 0);
}

template <bool BF16>
cudaError_t bwd_any(const BwdArgs& a) {
  constexpr int kSize = BF16 ? 2 : 4, VEC = 16 / kSize;
  // at most 16 elements a thread: two sums for each stay in registers
  constexpr int kBig = BF16 ? 2 : 4;
  LnShape sh;
  bool edge = false;
  int mis = 0;
  const void* const ptrs[] = {a.x, a.dy, a.dx};
  const int64_t lds[] = {a.ldx, a.lddy, a.cols};
  const bool vec = a.cols <= kLnMaxCols &&
                   vector_rows(ptrs, lds, 3, a.cols, kSize, &edge, &mis);
  const int64_t nvec = (a.cols + VEC - 1) / VEC + (edge ? 1 : 0);
  // several rows at a time where a row fits and there are rows for every SM
  // (rows off the boundary: a row at a time, 32 against 36 us at 5000 x 2563)
  if (vec && !edge && nvec <= 32 * kLnRowWarps && a.rows >= 4 * int64_t(sm_count()))
    return bwd_rows_any<BF16>(a, nvec);
  if (vec && ln_shape(nvec, kBig, a.rows, kLnBwdWarps, &sh)) {
    const bool multi = sh.split.W * sh.split.CS > 1;
    if (sh.nv == 1)
      return multi ? bwd_nv<BF16, 1, true>(a, sh, edge, mis)
                   : bwd_nv<BF16, 1, false>(a, sh, edge, mis);
    return multi ? bwd_nv<BF16, kBig, true>(a, sh, edge, mis)
                 : bwd_nv<BF16, kBig, false>(a, sh, edge, mis);
  }
  auto kern = k_ln_bwd_wide<BF16>;
  const int grid =
      persistent_grid(reinterpret_cast<const void*>(kern), kLnGenThreads, 0, a.rows);
  kern<<<grid, kLnGenThreads, 0, a.s>>>(a.dy, a.x, a.rows, a.cols, a.lddy, a.ldx, a.weight,
                                        a.mean, a.rstd, a.dx);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.dw == nullptr) return e;
  const int n = int(a.rows < kLnWidePartials ? a.rows : kLnWidePartials);
  k_ln_bwd_wide_params<BF16><<<dim3(unsigned((a.cols + 255) / 256), unsigned(n)), 256, 0, a.s>>>(
      a.dy, a.x, a.rows, a.cols, a.lddy, a.ldx, a.mean, a.rstd, a.partial);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : params_launch(a, n);
}

}  // namespace

cudaError_t launch_layernorm(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                             const float* weight, const float* bias, float eps, void* y,
                             float* mean, float* rstd, uint8_t* codes, uint8_t* scales,
                             cudaStream_t s) {
  const FwdArgs a = {x, rows, cols, ldx, weight, bias, eps, y, mean, rstd, codes, scales, s};
  return bf16 ? fwd_any<true>(a) : fwd_any<false>(a);
}

int64_t layernorm_backward_partials(int64_t rows) {
  return rows < kLnMaxPartials ? rows : kLnMaxPartials;
}

cudaError_t launch_layernorm_backward(const void* dy, const void* x, bool bf16, int64_t rows,
                                      int64_t cols, int64_t lddy, int64_t ldx,
                                      const float* weight, const float* mean, const float* rstd,
                                      void* dx, float* dw, float* db, float* partial,
                                      cudaStream_t s) {
  const BwdArgs a = {dy, x, rows, cols, lddy, ldx, weight, mean, rstd, dx, dw, db, partial, s};
  return bf16 ? bwd_any<true>(a) : bwd_any<false>(a);
}

}  // namespace mxfp4
