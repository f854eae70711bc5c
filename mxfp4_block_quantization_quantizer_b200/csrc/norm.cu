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
// writes dx, once each. A row lives in the registers of W warps (E = VEC NV
// elements a thread); the next row's loads are issued before this row's
// reductions, so loads stay in flight across them. Every statistic is fp32:
// each warp takes its own mean first and sums squares around it, and the
// warps' pairs (sum, squares) are joined with the exact correction
// n_w (mean_w - mean)^2, so a large common offset costs no precision.
// Persistent grid: the W warps keep their columns from row to row, so w and b
// stay in registers, and so do the column sums of the backward pass (for
// wide rows, in shared memory); each CTA writes one partial row of dw and db
// and a second small kernel adds those in a fixed order (no atomics: the
// same inputs give the same bits).
#include "launch.cuh"
#include "mxfp4_device.cuh"

namespace mxfp4 {

namespace {

constexpr int kLnMaxWarps = 16;      // warps that share a row
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

// A vector of VEC elements as loaded (16 bytes, or one element for rows that
// are not 16-byte aligned), and its fp32 pairs. A single element fills the
// low half of one pair; its high half stays zero and is never counted.
template <bool BF16, int VEC>
struct Vec;
template <>
struct Vec<true, 8> {
  static constexpr int kPairs = 4;
  uint4 r;
  __device__ __forceinline__ void load(const void* base, int64_t e) {
    r = ld_stream(static_cast<const uint16_t*>(base) + e);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(F2* p) const {
    p[0] = f2(bf16_lo(r.x), bf16_hi(r.x)), p[1] = f2(bf16_lo(r.y), bf16_hi(r.y));
    p[2] = f2(bf16_lo(r.z), bf16_hi(r.z)), p[3] = f2(bf16_lo(r.w), bf16_hi(r.w));
  }
  __device__ __forceinline__ void pack(const F2* p) {
    r = make_uint4(pack_bf16x2(f2_lo(p[0]), f2_hi(p[0])), pack_bf16x2(f2_lo(p[1]), f2_hi(p[1])),
                   pack_bf16x2(f2_lo(p[2]), f2_hi(p[2])), pack_bf16x2(f2_lo(p[3]), f2_hi(p[3])));
  }
  __device__ __forceinline__ void store(void* base, int64_t e) const {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e), r);
  }
};
template <>
struct Vec<false, 4> {
  static constexpr int kPairs = 2;
  uint4 r;
  __device__ __forceinline__ void load(const void* base, int64_t e) {
    r = ld_stream(static_cast<const float*>(base) + e);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(F2* p) const {
    p[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
    p[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  __device__ __forceinline__ void pack(const F2* p) {
    r = make_uint4(__float_as_uint(f2_lo(p[0])), __float_as_uint(f2_hi(p[0])),
                   __float_as_uint(f2_lo(p[1])), __float_as_uint(f2_hi(p[1])));
  }
  __device__ __forceinline__ void store(void* base, int64_t e) const {
    __stcs(reinterpret_cast<uint4*>(static_cast<float*>(base) + e), r);
  }
};
template <bool BF16>
struct Vec<BF16, 1> {
  static constexpr int kPairs = 1;
  uint32_t r;  // fp32 bits
  __device__ __forceinline__ void load(const void* base, int64_t e) {
    r = BF16 ? uint32_t(__ldg(static_cast<const uint16_t*>(base) + e)) << 16
             : __ldg(static_cast<const uint32_t*>(base) + e);
  }
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ void unpack(F2* p) const { p[0] = f2(__uint_as_float(r), 0.0f); }
  __device__ __forceinline__ void pack(const F2* p) {
    r = BF16 ? pack_bf16x2(f2_lo(p[0]), 0.0f) : __float_as_uint(f2_lo(p[0]));
  }
  __device__ __forceinline__ void store(void* base, int64_t e) const {
    if (BF16)
      static_cast<uint16_t*>(base)[e] = uint16_t(r);
    else
      static_cast<uint32_t*>(base)[e] = r;
  }
};

// VEC fp32 parameters of columns e .. e + VEC - 1 (16-byte aligned where
// VEC > 1) as pairs; `fill` where there is no parameter tensor.
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, int64_t e, float fill, F2* out) {
  if constexpr (VEC == 1) {
    out[0] = f2(p != nullptr ? __ldg(p + e) : fill, 0.0f);
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      float4 v = make_float4(fill, fill, fill, fill);
      if (p != nullptr) v = __ldg(reinterpret_cast<const float4*>(p + e) + j);
      out[2 * j] = f2(v.x, v.y), out[2 * j + 1] = f2(v.z, v.w);
    }
  }
}

// The same for VEC fp32 values in shared memory.
template <int VEC>
__device__ __forceinline__ void load_shared(const float* p, F2* out) {
  if constexpr (VEC == 1) {
    out[0] = f2(*p, 0.0f);
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const float4 v = reinterpret_cast<const float4*>(p)[j];
      out[2 * j] = f2(v.x, v.y), out[2 * j + 1] = f2(v.z, v.w);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void store_shared(float* p, const F2* in) {
  if constexpr (VEC == 1) {
    *p = f2_lo(in[0]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j)
      reinterpret_cast<float4*>(p)[j] =
          make_float4(f2_lo(in[2 * j]), f2_hi(in[2 * j]), f2_lo(in[2 * j + 1]),
                      f2_hi(in[2 * j + 1]));
  }
}

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

// v^-1/2 to an ulp: the approximation and one Newton step.
__device__ __forceinline__ float rsqrt_exact(float v) {
  const float r = rsqrtf(v);
  const float e = __fmaf_rn(-__fmul_rn(v, r), r, 1.0f);
  const float n = __fmaf_rn(__fmul_rn(0.5f, r), e, r);
  return v > 0.0f && v < __uint_as_float(0x7F800000u) ? n : r;
}

// Barrier of the W warps of row group g (id 1 + g), or of one warp.
__device__ __forceinline__ void group_sync(int g, int W) {
  if (W == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(W * 32) : "memory");
}

// Where a thread stands: the W warps of group g take whole rows; thread t of
// them holds vectors t, t + 32 W, ... of the row's nvec.
struct Place {
  int W, P, g, G, w, lane, t;
};
__device__ __forceinline__ Place place(int W, int P) {
  Place p;
  p.W = W, p.P = P;
  const int warp = threadIdx.x >> 5;
  p.g = warp / W, p.G = (blockDim.x >> 5) / W;
  p.w = warp % W, p.lane = threadIdx.x & 31;
  p.t = p.w * 32 + p.lane;
  return p;
}

// Forward. QUANT also (or only) writes the 1x32 codes and scales of the
// rounded y: a group is 32 / VEC adjacent lanes (rows are 16-byte aligned
// and cols is a multiple of 32, so a group never splits over warps).
template <bool BF16, int VEC, int NV, bool QUANT>
__global__ void __launch_bounds__(512)
    k_ln_fwd(const void* __restrict__ x, int64_t rows, int cols, int64_t ldx,
             const float* __restrict__ weight, const float* __restrict__ bias, float eps,
             void* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
             uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int W, int P) {
  using V = Vec<BF16, VEC>;
  constexpr int NP = V::kPairs;
  // w and b stay in registers where the row's share leaves room for them
  constexpr bool kKeep = VEC * NV <= (BF16 ? 24 : 16);
  __shared__ float2 red[2][kLnMaxWarps];
  const Place p = place(W, P);
  const int nvec = cols / VEC, step = 32 * W;
  const int64_t stride = int64_t(gridDim.x) * p.G;
  const float inv_n = __fdiv_rn(1.0f, float(cols));

  // valid elements of this warp, and of warp `lane` of the group
  float my_n = 0.0f, lane_n = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    my_n += float(min(max(nvec - i * step - p.w * 32, 0), 32) * VEC);
    lane_n += float(min(max(nvec - i * step - p.lane * 32, 0), 32) * VEC);
  }
  const float my_inv = my_n > 0.0f ? __fdiv_rn(1.0f, my_n) : 0.0f;
  const float lane_inv = lane_n > 0.0f && p.lane < W ? __fdiv_rn(1.0f, lane_n) : 0.0f;

  F2 wk[kKeep ? NV * NP : 1], bk[kKeep ? NV * NP : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.t + i * step;
      if (v < nvec) {
        load_param<VEC>(weight, int64_t(v) * VEC, 1.0f, wk + i * NP);
        load_param<VEC>(bias, int64_t(v) * VEC, 0.0f, bk + i * NP);
      } else {
#pragma unroll
        for (int j = 0; j < NP; ++j) wk[i * NP + j] = bk[i * NP + j] = f2(0.0f, 0.0f);
      }
    }
  }

  V nx[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.t + i * step;
      if (row < rows && v < nvec)
        nx[i].load(x, row * ldx + int64_t(v) * VEC);
      else
        nx[i].zero();
    }
  };
  int64_t row = int64_t(blockIdx.x) * p.G + p.g;
  fetch(row);
  for (int par = 0; row < rows; row += stride, par ^= 1) {
    F2 a[NV * NP];
#pragma unroll
    for (int i = 0; i < NV; ++i) nx[i].unpack(a + i * NP);
    fetch(row + stride);
    F2 s2 = f2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV * NP; ++i) s2 = add2(s2, a[i]);
    const float s = warp_sum(__fadd_rn(f2_lo(s2), f2_hi(s2)));
    float mean = __fmul_rn(s, my_inv);
    F2 q2 = f2(0.0f, 0.0f);
    const F2 mm = VEC == 1 ? f2(-mean, 0.0f) : f2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (p.t + i * step < nvec) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const F2 d = add2(a[i * NP + j], mm);
          q2 = fma2(d, d, q2);
        }
      }
    float m2 = warp_sum(__fadd_rn(f2_lo(q2), f2_hi(q2)));
    if (W > 1) {
      // one barrier a row: the buffer of this parity is written again two
      // rows on, past the next row's barrier
      float2* rd = red[par];
      if (p.lane == 0) rd[p.g * W + p.w] = make_float2(s, m2);
      group_sync(p.g, W);
      const int l = p.lane & (P - 1);
      const float2 o = l < W ? rd[p.g * W + l] : make_float2(0.0f, 0.0f);
      mean = __fmul_rn(part_sum(o.x, P), inv_n);
      const float ln = __shfl_sync(0xFFFFFFFFu, lane_n, l);
      const float li = __shfl_sync(0xFFFFFFFFu, lane_inv, l);
      const float d = __fsub_rn(__fmul_rn(o.x, li), mean);
      m2 = part_sum(l < W ? __fmaf_rn(__fmul_rn(ln, d), d, o.y) : 0.0f, P);
    }
    const float rstd = rsqrt_exact(__fmaf_rn(m2, inv_n, eps));
    if (p.t == 0) {
      if (mean_out != nullptr) mean_out[row] = mean;
      if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
    const F2 nm = f2(-mean, -mean), rs = f2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.t + i * step;
      const bool in = v < nvec;
      if (!QUANT && !in) continue;
      F2 o[NP];
      F2 wl[NP], bl[NP];
      if constexpr (!kKeep) {
        if (in) {
          load_param<VEC>(weight, int64_t(v) * VEC, 1.0f, wl);
          load_param<VEC>(bias, int64_t(v) * VEC, 0.0f, bl);
        } else {
#pragma unroll
          for (int j = 0; j < NP; ++j) wl[j] = bl[j] = f2(0.0f, 0.0f);
        }
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const F2 h = mul2(add2(a[i * NP + j], nm), rs);
        o[j] = fma2(h, kKeep ? wk[kKeep ? i * NP + j : 0] : wl[j],
                    kKeep ? bk[kKeep ? i * NP + j : 0] : bl[j]);
      }
      V out;
      out.pack(o);
      if (in && y != nullptr) out.store(y, row * cols + int64_t(v) * VEC);
      if constexpr (QUANT && VEC > 1) {
        const int64_t e = row * cols + int64_t(v) * VEC;
        if constexpr (BF16) {
          uint32_t am = bf16x8_absmax(out.r);
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          const uint32_t sb = scale_byte(am);
          const float mul = inv_scale(sb);
          float qv[8];
          F2 r8[4];
          out.unpack(r8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            qv[2 * j] = __fmul_rn(f2_lo(r8[j]), mul);
            qv[2 * j + 1] = __fmul_rn(f2_hi(r8[j]), mul);
          }
          const uint32_t word = sb == 0xFFu ? 0u : e2m1x8_rn(qv);
          if (in) {
            *reinterpret_cast<uint32_t*>(codes + e / 2) = word;
            if ((p.lane & 3) == 0) scales[e / 32] = static_cast<uint8_t>(sb);
          }
        } else {
          uint32_t am = max(max(out.r.x & 0x7FFFFFFFu, out.r.y & 0x7FFFFFFFu),
                            max(out.r.z & 0x7FFFFFFFu, out.r.w & 0x7FFFFFFFu));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 4));
          const uint32_t sb = scale_byte(am);
          const float mul = inv_scale(sb);
          const float qv[8] = {__fmul_rn(__uint_as_float(out.r.x), mul),
                               __fmul_rn(__uint_as_float(out.r.y), mul),
                               __fmul_rn(__uint_as_float(out.r.z), mul),
                               __fmul_rn(__uint_as_float(out.r.w), mul), 0, 0, 0, 0};
          const uint32_t word = sb == 0xFFu ? 0u : e2m1x8_rn(qv);
          if (in) {
            *reinterpret_cast<uint16_t*>(codes + e / 2) = static_cast<uint16_t>(word);
            if ((p.lane & 7) == 0) scales[e / 32] = static_cast<uint8_t>(sb);
          }
        }
      }
    }
  }
}

// Rows wider than the registers of 16 warps: one CTA a row, three passes
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

// Backward. SMACC keeps the column sums of dw and db in shared memory
// ([2][cols] floats) instead of registers; PARAMS = false leaves them out.
template <bool BF16, int VEC, int NV, bool SMACC, bool PARAMS>
__global__ void __launch_bounds__(512)
    k_ln_bwd(const void* __restrict__ dy, const void* __restrict__ x, int64_t rows, int cols,
             int64_t lddy, int64_t ldx, const float* __restrict__ weight,
             const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
             void* __restrict__ dx, float* __restrict__ partial, int W, int P) {
  using V = Vec<BF16, VEC>;
  constexpr int NP = V::kPairs;
  constexpr bool kRegAcc = PARAMS && !SMACC;
  constexpr bool kKeep = !SMACC;  // the weight's columns in registers
  extern __shared__ __align__(16) float sacc[];
  __shared__ float2 red[2][kLnMaxWarps];
  const Place p = place(W, P);
  const int nvec = cols / VEC, step = 32 * W;
  const int64_t stride = int64_t(gridDim.x) * p.G;
  const float inv_n = __fdiv_rn(1.0f, float(cols));
  const F2 zero = f2(0.0f, 0.0f);

  F2 wk[kKeep ? NV * NP : 1];
  F2 aw[kRegAcc ? NV * NP : 1], ab[kRegAcc ? NV * NP : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = p.t + i * step;
    if constexpr (kKeep) {
      if (v < nvec) {
        load_param<VEC>(weight, int64_t(v) * VEC, 1.0f, wk + i * NP);
      } else {
#pragma unroll
        for (int j = 0; j < NP; ++j) wk[i * NP + j] = zero;
      }
    }
    if constexpr (kRegAcc) {
#pragma unroll
      for (int j = 0; j < NP; ++j) aw[i * NP + j] = ab[i * NP + j] = zero;
    }
    if constexpr (PARAMS && SMACC) {
      if (v < nvec) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          sacc[v * VEC + j] = 0.0f;
          sacc[cols + v * VEC + j] = 0.0f;
        }
      }
    }
  }

  V nx[NV], ny[NV];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row < rows) nmean = __ldg(mean_in + row), nrstd = __ldg(rstd_in + row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.t + i * step;
      if (row < rows && v < nvec) {
        nx[i].load(x, row * ldx + int64_t(v) * VEC);
        ny[i].load(dy, row * lddy + int64_t(v) * VEC);
      } else {
        nx[i].zero(), ny[i].zero();
      }
    }
  };
  int64_t row = int64_t(blockIdx.x) * p.G + p.g;
  fetch(row);
  for (int par = 0; row < rows; row += stride, par ^= 1) {
    F2 h[NV * NP], g[NV * NP];
    const float mean = nmean, rstd = nrstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) nx[i].unpack(h + i * NP), ny[i].unpack(g + i * NP);
    fetch(row + stride);
    const F2 nm = f2(-mean, -mean), rs = f2(rstd, rstd);
    F2 c1 = zero, c2 = zero;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.t + i * step;
      if (v >= nvec) continue;
      F2 wl[NP], sw[NP], sb[NP];
      if constexpr (!kKeep) load_param<VEC>(weight, int64_t(v) * VEC, 1.0f, wl);
      if constexpr (PARAMS && SMACC) {
        load_shared<VEC>(sacc + v * VEC, sw);
        load_shared<VEC>(sacc + cols + v * VEC, sb);
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int k = i * NP + j;
        h[k] = mul2(add2(h[k], nm), rs);
        if constexpr (kRegAcc) {
          aw[k] = fma2(g[k], h[k], aw[k]);
          ab[k] = add2(ab[k], g[k]);
        }
        if constexpr (PARAMS && SMACC) {
          sw[j] = fma2(g[k], h[k], sw[j]);
          sb[j] = add2(sb[j], g[k]);
        }
        g[k] = mul2(g[k], kKeep ? wk[kKeep ? k : 0] : wl[j]);
        c1 = add2(c1, g[k]);
        c2 = fma2(g[k], h[k], c2);
      }
      if constexpr (PARAMS && SMACC) {
        store_shared<VEC>(sacc + v * VEC, sw);
        store_shared<VEC>(sacc + cols + v * VEC, sb);
      }
    }
    // the high half of a single element's pair is padding
    float s1 = warp_sum(VEC == 1 ? f2_lo(c1) : __fadd_rn(f2_lo(c1), f2_hi(c1)));
    float s2 = warp_sum(VEC == 1 ? f2_lo(c2) : __fadd_rn(f2_lo(c2), f2_hi(c2)));
    if (W > 1) {
      float2* rd = red[par];
      if (p.lane == 0) rd[p.g * W + p.w] = make_float2(s1, s2);
      group_sync(p.g, W);
      const int l = p.lane & (P - 1);
      const float2 o = l < W ? rd[p.g * W + l] : make_float2(0.0f, 0.0f);
      s1 = part_sum(o.x, P);
      s2 = part_sum(o.y, P);
    }
    const float m1 = -__fmul_rn(s1, inv_n), m2 = -__fmul_rn(s2, inv_n);
    const F2 k1 = f2(m1, m1), k2 = f2(m2, m2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = p.t + i * step;
      if (v >= nvec) continue;
      F2 o[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int k = i * NP + j;
        o[j] = mul2(add2(fma2(h[k], k2, g[k]), k1), rs);
      }
      V out;
      out.pack(o);
      out.store(dx, row * cols + int64_t(v) * VEC);
    }
  }

  if constexpr (PARAMS) {
    float* pw = partial + int64_t(blockIdx.x) * 2 * cols;
    if constexpr (SMACC) {
      // one group a CTA: every thread writes the columns it summed
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = p.t + i * step;
        if (v >= nvec) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          pw[v * VEC + j] = sacc[v * VEC + j];
          pw[cols + v * VEC + j] = sacc[cols + v * VEC + j];
        }
      }
    } else {
      // the groups of a CTA add into shared memory one after the other (the
      // last writes the partial row)
      for (int g = 0; g < p.G; ++g) {
        if (g > 0) __syncthreads();
        if (p.g != g) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = p.t + i * step;
          if (v >= nvec) continue;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float a = (j & 1) ? f2_hi(aw[i * NP + j / 2]) : f2_lo(aw[i * NP + j / 2]);
            float b = (j & 1) ? f2_hi(ab[i * NP + j / 2]) : f2_lo(ab[i * NP + j / 2]);
            const int c = v * VEC + j;
            if (g > 0) a = __fadd_rn(a, sacc[c]), b = __fadd_rn(b, sacc[cols + c]);
            if (g + 1 == p.G)
              pw[c] = a, pw[cols + c] = b;
            else
              sacc[c] = a, sacc[cols + c] = b;
          }
        }
      }
    }
  }
}

// Rows wider than the registers of 16 warps: dx with one CTA a row, and the
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
  int nv, W, P, G, threads;
};

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// The number of vectors a thread holds (one of `nvs`, ascending) and the
// warps W of a row: the preferred count `want` unless the row needs more;
// few rows (less than two an SM) take the smallest count, which spreads a
// row over the most threads. Narrow rows share a CTA of about 8 warps.
bool ln_shape(int64_t cols, int vec, const int* nvs, int n_nvs, int want, int64_t rows,
              int block_warps, LnShape* s) {
  if (cols % vec != 0) return false;
  const int64_t nvec = cols / vec;
  const bool few = rows < 2 * int64_t(sm_count());
  for (int i = 0; i < n_nvs; ++i) {
    const int64_t W = (nvec + 32 * nvs[i] - 1) / (32 * nvs[i]);
    if (W > kLnMaxWarps) continue;
    if (!few && nvs[i] < want && i + 1 < n_nvs && W > 1) continue;
    s->nv = nvs[i];
    s->W = int(W);
    s->P = 1;
    while (s->P < s->W) s->P *= 2;
    s->G = few ? 1 : (block_warps / s->W > 1 ? block_warps / s->W : 1);
    s->threads = 32 * s->W * s->G;
    return true;
  }
  return false;
}

bool aligned_rows(const void* p, int64_t ld, int size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
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

template <bool BF16, int VEC, int NV, bool QUANT>
cudaError_t fwd_launch(const FwdArgs& a, const LnShape& sh) {
  auto kern = k_ln_fwd<BF16, VEC, NV, QUANT>;
  const int grid = persistent_grid(reinterpret_cast<const void*>(kern), sh.threads, 0,
                                   (a.rows + sh.G - 1) / sh.G);
  kern<<<grid, sh.threads, 0, a.s>>>(a.x, a.rows, int(a.cols), a.ldx, a.weight, a.bias, a.eps,
                                     a.y, a.mean, a.rstd, a.codes, a.scales, sh.W, sh.P);
  return cudaGetLastError();
}

template <bool BF16, bool QUANT>
cudaError_t fwd_vec(const FwdArgs& a, const LnShape& sh) {
  constexpr int VEC = BF16 ? 8 : 4;
  switch (sh.nv) {
    case 1: return fwd_launch<BF16, VEC, 1, QUANT>(a, sh);
    case 2: return fwd_launch<BF16, VEC, 2, QUANT>(a, sh);
    case 3: return fwd_launch<BF16, VEC, 3, QUANT>(a, sh);
    case 4: return fwd_launch<BF16, VEC, 4, QUANT>(a, sh);
    default: return fwd_launch<BF16, VEC, 8, QUANT>(a, sh);
  }
}

template <bool BF16>
cudaError_t fwd_any(const FwdArgs& a) {
  constexpr int kSize = BF16 ? 2 : 4, VEC = 16 / kSize;
  static const int bf_nvs[] = {1, 2, 3, 4}, f_nvs[] = {1, 2, 4, 8}, one_nvs[] = {8, 16, 32};
  LnShape sh;
  const bool vec = a.cols % VEC == 0 && aligned_rows(a.x, a.ldx, kSize) &&
                   (a.y == nullptr || aligned_rows(a.y, a.cols, kSize)) &&
                   aligned_rows(a.weight, 0, 4) && aligned_rows(a.bias, 0, 4);
  if (vec && ln_shape(a.cols, VEC, BF16 ? bf_nvs : f_nvs, 4, BF16 ? 3 : 4, a.rows, 8, &sh))
    return a.codes != nullptr ? fwd_vec<BF16, true>(a, sh) : fwd_vec<BF16, false>(a, sh);
  if (a.codes == nullptr && ln_shape(a.cols, 1, one_nvs, 3, 16, a.rows, 8, &sh)) {
    switch (sh.nv) {
      case 8: return fwd_launch<BF16, 1, 8, false>(a, sh);
      case 16: return fwd_launch<BF16, 1, 16, false>(a, sh);
      default: return fwd_launch<BF16, 1, 32, false>(a, sh);
    }
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

template <bool BF16, int VEC, int NV, bool SMACC, bool PARAMS>
cudaError_t bwd_launch(const BwdArgs& a, const LnShape& sh) {
  auto kern = k_ln_bwd<BF16, VEC, NV, SMACC, PARAMS>;
  const size_t smem = PARAMS && (SMACC || sh.G > 1) ? size_t(a.cols) * 8 : 0;
  if (smem > 0) {
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
  }
  int64_t blocks = (a.rows + sh.G - 1) / sh.G;
  if (blocks > kLnMaxPartials) blocks = kLnMaxPartials;
  const int grid = persistent_grid(reinterpret_cast<const void*>(kern), sh.threads, smem, blocks);
  kern<<<grid, sh.threads, smem, a.s>>>(a.dy, a.x, a.rows, int(a.cols), a.lddy, a.ldx, a.weight,
                                        a.mean, a.rstd, a.dx, a.partial, sh.W, sh.P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !PARAMS) return e;
  return params_launch(a, grid);
}

template <bool BF16, int VEC, int NV, bool SMACC>
cudaError_t bwd_params(const BwdArgs& a, const LnShape& sh) {
  return a.dw != nullptr ? bwd_launch<BF16, VEC, NV, SMACC, true>(a, sh)
                         : bwd_launch<BF16, VEC, NV, SMACC, false>(a, sh);
}

template <bool BF16>
cudaError_t bwd_any(const BwdArgs& a) {
  constexpr int kSize = BF16 ? 2 : 4, VEC = 16 / kSize;
  static const int bf_nvs[] = {1, 2, 4}, f_nvs[] = {2, 4, 8}, one_nvs[] = {8, 16, 32};
  LnShape sh;
  const bool vec = a.cols % VEC == 0 && aligned_rows(a.x, a.ldx, kSize) &&
                   aligned_rows(a.dy, a.lddy, kSize) && aligned_rows(a.dx, a.cols, kSize) &&
                   aligned_rows(a.weight, 0, 4);
  if (vec && ln_shape(a.cols, VEC, BF16 ? bf_nvs : f_nvs, 3, BF16 ? 2 : 4, a.rows, 4, &sh)) {
    if constexpr (BF16) {
      switch (sh.nv) {
        case 1: return bwd_params<BF16, VEC, 1, false>(a, sh);
        case 2: return bwd_params<BF16, VEC, 2, false>(a, sh);
        default: return bwd_params<BF16, VEC, 4, true>(a, sh);
      }
    } else {
      switch (sh.nv) {
        case 2: return bwd_params<BF16, VEC, 2, false>(a, sh);
        case 4: return bwd_params<BF16, VEC, 4, false>(a, sh);
        default: return bwd_params<BF16, VEC, 8, true>(a, sh);
      }
    }
  }
  if (ln_shape(a.cols, 1, one_nvs, 3, 8, a.rows, 4, &sh)) {
    switch (sh.nv) {
      case 8: return bwd_params<BF16, 1, 8, false>(a, sh);
      case 16: return bwd_params<BF16, 1, 16, true>(a, sh);
      default: return bwd_params<BF16, 1, 32, true>(a, sh);
    }
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
