// Newton-Schulz orthogonalization of a weight's update (sm_100a).
//
//   X = G / (|G|_F + eps);  repeat: A = X X^T, B = b A + c A A, X = a X + B X
// (for more rows than columns A = X^T X and X = a X + X B, the same numbers).
// Every singular value s of X moves to a s + b s^3 + c s^5, towards 1, while
// the singular vectors stay.
//
// Bound by the tensor cores: with s <= l the sides, a step costs s s l flops
// for A (half of a symmetric product), s^3 for A A (half) and 2 s s l for
// B X. Three products a step, each a persistent tcgen05 GEMM with a fused
// epilogue; only the tiles on and above the diagonal of A and B are computed
// and written to both sides. (The sums of a tile stay in one accumulator: four
// that a stage's MMAs took in turn made small products 2 to 5% slower.) Small
// matrices are bound by the latency of launches that depend on one another,
// about 5 us each (256 x 512, five steps, 17 launches: 82 us); each may set
// itself up while the one before it ends. A short side of few tiles with a
// long one leaves A to few SMs, which walk all of K (128 x 14336: 225 us).
// Large ones: 4096 x 14336, five steps, 3.1 to 3.5 ms in a short run, 3.6 to
// 3.9 ms where the GPU has reached its power limit: 1.27 to 1.01 PFLOP/s of
// the flops above.
//
// Numbers: operands are fp16, not bf16, at the same tensor rate and with
// three more significant bits. Their range suffices because everything here
// is bounded (singular values of X below about 1.2): X, A and B are stored
// times 2^12, where entries up to 15.9 fit and entries from 2^-26 up keep
// all their bits. X itself is carried as two fp16 values (hi + lo, about 22
// bits): a X in the epilogue uses both, the products use hi. With the carry
// rounded to fp16 the error of five steps on a matrix with strong and weak
// directions (rank 64 plus noise 20 times smaller, 512 x 512) is 4.8e-3 of
// the result, with both halves 3.9e-4; with bf16 operands and carry 5.9e-2.
// Sums are fp32 in tensor memory, the norm's in fp64.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "mxfp4_device.cuh"
#include "tc_common.cuh"

namespace mxfp4 {

namespace {

constexpr float kNsScale = 4096.0f, kNsInv = 1.0f / 4096.0f;
constexpr int kSM = 128;            // tile rows
constexpr int kSK = 64;             // K elements of a stage: one swizzle row
constexpr int kSEpiWarps = 8;
constexpr int kSThreads = 32 * (3 + kSEpiWarps);  // A loads, MMA, epilogue, B loads
constexpr int kSLoadB = 2 + kSEpiWarps;           // the warp of the B loads
constexpr int kNsPartials = 592;    // partial sums of the norm
constexpr int64_t kNsPairTiles = 120;  // fewest tiles for CTA pairs

// What a product's epilogue does.
enum NsMode { kGram = 0, kSquare = 1, kStep = 2, kLast = 3 };

struct NsArgs {
  int64_t m, n, k;      // product: [m][k] x [n][k]
  int64_t ldd;          // pitch of c_hi, c_lo, d_hi, d_lo (elements)
  float alpha, beta;    // D = alpha acc + beta C, all times 2^12
  const __half *c_hi, *c_lo;
  __half *d_hi, *d_lo;
  void* out;            // kLast: [m][n] of the caller's type
  int out_bf16, out_vec;  // out_vec: rows of out are whole 16-byte vectors of 8
  float out_scale;
  int* status;
};

template <int BN>
struct NsLayout {
  static constexpr int kStages = BN == 128 ? 6 : 8;
  static constexpr uint32_t kA = kSM * 128, kB = BN * 128;
  static constexpr uint32_t kBOff = kStages * kA;
  // per epilogue warp: 32 rows x 32 fp16, rows 80 bytes apart (no bank twice)
  static constexpr uint32_t kEpiOff = kBOff + kStages * kB;
  static constexpr uint32_t kBarOff = kEpiOff + kSEpiWarps * 32 * 80;
  static constexpr uint32_t kBytes = kBarOff + 256;
  static constexpr uint32_t kTmemCols = 2 * BN;  // two accumulators
  // kind::f16: fp32 accumulator, fp16 operands (0), majorness bits 15, 16
  __host__ __device__ static constexpr uint32_t idesc(bool a_mn, bool b_mn) {
    return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(BN >> 3) << 17) | (uint32_t(kSM >> 4) << 24);
  }
};

__device__ __forceinline__ void mma_f16(uint32_t tmem_c, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_c),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// Descriptor of an operand stored with K along the rows of shared memory
// (MN-major): boxes of 64 MN elements (128 bytes, 128-byte swizzle) x 64 K
// rows; 8-row groups 1024 bytes apart, boxes 8192 bytes apart. A K step of
// 16 moves the start by 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn(const void* p) {
  uint64_t d = (smem_u32(p) >> 4) & 0x3FFFu;
  d |= uint64_t(8192 >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// Tile `t` of the order that all roles walk. Full products: groups of 16 row
// tiles swept across all column tiles (their panels stay in L2). Symmetric
// products: the tiles that reach the diagonal or above, column by column
// (narrow tiles: row by row).
template <int BN, bool SYM>
__device__ __forceinline__ void ns_tile(int64_t t, int64_t mt, int64_t nt, int64_t& m0,
                                        int64_t& n0) {
  if constexpr (SYM) {
    // row tile i starts at column tile i * 128 / BN
    if constexpr (BN >= kSM) {
      constexpr int R = BN / kSM;  // row tiles per column tile
      int64_t j = nt - 1;
      for (; j > 0; --j) {
        const int64_t rows = (j + 1) * R < mt ? (j + 1) * R : mt;
        if (t < rows) break;
        t -= rows;
      }
      n0 = j * BN, m0 = t * kSM;
    } else {
      constexpr int R = kSM / BN;  // column tiles per row tile
      int64_t i = 0;
      for (; i < mt - 1; ++i) {
        const int64_t cols = nt - i * R;
        if (t < cols) break;
        t -= cols;
      }
      m0 = i * kSM, n0 = (i * R + t) * BN;
    }
  } else {
    constexpr int64_t G = 16;
    const int64_t per = G * nt, g = t / per, r = t % per;
    const int64_t gm = mt - g * G < G ? mt - g * G : G;
    m0 = (g * G + r % gm) * kSM;
    n0 = (r / gm) * BN;
  }
}
template <int BN>
__host__ __device__ inline int64_t ns_tiles(bool sym, int64_t mt, int64_t nt) {
  if (!sym) return mt * nt;
  int64_t n = 0;
  if (BN >= kSM) {
    for (int64_t j = 0; j < nt; ++j) {
      const int64_t rows = (j + 1) * (BN / kSM);
      n += rows < mt ? rows : mt;
    }
  } else {
    for (int64_t i = 0; i < mt; ++i) n += nt - i * (kSM / BN);
  }
  return n;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

#define MXFP4_TMEM_LD32(d, addr)                                                               \
  asm volatile(                                                                                \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, "                   \
      "%7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "                    \
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"                         \
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]),    \
        "=r"(d[7]), "=r"(d[8]), "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]),             \
        "=r"(d[13]), "=r"(d[14]), "=r"(d[15]), "=r"(d[16]), "=r"(d[17]), "=r"(d[18]),          \
        "=r"(d[19]), "=r"(d[20]), "=r"(d[21]), "=r"(d[22]), "=r"(d[23]), "=r"(d[24]),          \
        "=r"(d[25]), "=r"(d[26]), "=r"(d[27]), "=r"(d[28]), "=r"(d[29]), "=r"(d[30]),          \
        "=r"(d[31])                                                                            \
      : "r"(addr))

// Lane l of a warp holds row l of a 32 x 32 tile in v[0..31]; afterwards it
// holds column l.
__device__ __forceinline__ void transpose32(float* v, int lane) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j & s) continue;
      const float give = up ? v[j] : v[j + s];
      const float got = __shfl_xor_sync(0xFFFFFFFFu, give, s);
      if (up)
        v[j] = got;
      else
        v[j + s] = got;
    }
  }
}

// Store a warp's 32 x 32 fp16 tile, lane l holding row l in w[0..15]: through
// the warp's staging tile, so that an instruction writes 8 rows of 64 bytes
// and not 32 of 16 (which took the epilogue three times as long).
__device__ __forceinline__ void store_tile(uint8_t* stage, const uint32_t* w, __half* d,
                                           int64_t ldd, int64_t row0, int64_t c0, int64_t m,
                                           int64_t n) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<uint4*>(stage + lane * 80 + 16 * g) =
        make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
  __syncwarp();
  // (rows are padded to whole 16-byte chunks)
  const int64_t c = c0 + 8 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 80 + 16 * (lane & 3));
    if (row0 + r < m && c < n) *reinterpret_cast<uint4*>(d + (row0 + r) * ldd + c) = v;
  }
  __syncwarp();
}

// The epilogue of one warp for its row (lane) and the BN / 2 columns from n0
// on, in rounds of 32: waits for the products, reads them from tensor memory
// at `tb` and stores D. Returns false (and stores NaN) if the wait ran out.
template <int BN, int MODE, bool SYM>
__device__ __forceinline__ bool ns_epilogue(const NsArgs& p, int64_t row, int64_t n0, uint32_t tb,
                                            uint8_t* stage, unsigned long long* acc_full,
                                            uint32_t phase, int* failed) {
  constexpr int kCols = BN / 2;
  constexpr bool kHasC = MODE != kGram, kHasLo = MODE == kStep || MODE == kLast;
  // C's share of 32 columns, loaded a round ahead (the first one before the
  // products are done): one dependent load after the other took longer than
  // the main loop of a narrow tile
  struct Chunk {
    uint4 hi[4], lo[4];
  };
  auto fetch = [&](Chunk& f, int64_t c0) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      // rows are padded to whole 16-byte chunks
      const bool in = row < p.m && c0 + 8 * g < p.n;
      if (kHasC && in) f.hi[g] = __ldcg(reinterpret_cast<const uint4*>(p.c_hi + row * p.ldd + c0 + 8 * g));
      if (kHasLo && in) f.lo[g] = __ldcg(reinterpret_cast<const uint4*>(p.c_lo + row * p.ldd + c0 + 8 * g));
    }
  };
  Chunk cur, next;
#pragma unroll
  for (int g = 0; g < 4; ++g) cur.hi[g] = cur.lo[g] = make_uint4(0, 0, 0, 0);
  next = cur;
  if constexpr (kHasC) fetch(cur, n0);
  const bool ok = __all_sync(0xFFFFFFFFu, !failed_flag(failed) &&
                                              wait_parity(acc_full, phase, kAccWaitLimit));
  if (!ok) atomicExch(failed, 1);
  asm volatile("tcgen05.fence::after_thread_sync;");
#pragma unroll 1
  for (int cb = 0; cb < kCols; cb += 32) {
    uint32_t v[32];
    MXFP4_TMEM_LD32(v, tb + cb);
    const int64_t c0 = n0 + cb;
    if constexpr (kHasC)
      if (cb + 32 < kCols) fetch(next, c0 + 32);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    if (!ok || failed_flag(failed)) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0x7FC00000u;
    }
    float o[32];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[8 * g + j] = __fmul_rn(p.alpha, __uint_as_float(v[8 * g + j]));
      if constexpr (kHasC) {
        const uint32_t hw[4] = {cur.hi[g].x, cur.hi[g].y, cur.hi[g].z, cur.hi[g].w};
        const uint32_t lw[4] = {cur.lo[g].x, cur.lo[g].y, cur.lo[g].z, cur.lo[g].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 f = unpack_h2(hw[j]);
          if constexpr (kHasLo) {
            const float2 l = unpack_h2(lw[j]);
            f.x = __fadd_rn(f.x, l.x), f.y = __fadd_rn(f.y, l.y);
          }
          o[8 * g + 2 * j] = __fmaf_rn(p.beta, f.x, o[8 * g + 2 * j]);
          o[8 * g + 2 * j + 1] = __fmaf_rn(p.beta, f.y, o[8 * g + 2 * j + 1]);
        }
      }
    }
    if constexpr (MODE == kLast) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __fmul_rn(o[j], p.out_scale);
      if (p.out_vec) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t c = c0 + 8 * g;
          const float* e = o + 8 * g;
          if (row >= p.m || c >= p.n) continue;
          if (p.out_bf16) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.n + c) =
                make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]),
                           pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7]));
          } else {
            float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.n + c);
            to[0] = make_float4(e[0], e[1], e[2], e[3]);
            to[1] = make_float4(e[4], e[5], e[6], e[7]);
          }
        }
      } else {
        // rows off a 16-byte boundary: a lane takes a column, so that a warp
        // stores 32 neighbours at a time
        const int lane = threadIdx.x & 31;
        transpose32(o, lane);
        const int64_t c = c0 + lane, r0 = row - lane;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (r0 + j >= p.m || c >= p.n) continue;
          if (p.out_bf16)
            static_cast<uint16_t*>(p.out)[(r0 + j) * p.n + c] = uint16_t(pack_bf16x2(o[j], 0.0f));
          else
            static_cast<float*>(p.out)[(r0 + j) * p.n + c] = o[j];
        }
      }
    } else {
      const int64_t row0 = row - (threadIdx.x & 31);
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = pack_h2(o[2 * j], o[2 * j + 1]);
      if constexpr (SYM) {
        // each entry of the symmetric result has one writer, the element on
        // or above the diagonal, for both sides
        if (c0 >= row0 + 31) {
          store_tile(stage, w, p.d_hi, p.ldd, row0, c0, p.m, p.n);
        } else if (row < p.m) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c0 + j >= row && c0 + j < p.n)
              p.d_hi[row * p.ldd + c0 + j] =
                  __ushort_as_half(uint16_t(w[j / 2] >> (16 * (j & 1))));
        }
        if (row < p.m) {
          __half* to = p.d_hi + c0 * p.ldd + row;
#pragma unroll
          for (int j = 0; j < 32; ++j, to += p.ldd)
            if (c0 + j >= row && c0 + j < p.n)
              *to = __ushort_as_half(uint16_t(w[j / 2] >> (16 * (j & 1))));
        }
      } else {
        store_tile(stage, w, p.d_hi, p.ldd, row0, c0, p.m, p.n);
        if constexpr (kHasLo) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 f = unpack_h2(w[j]);
            w[j] = pack_h2(__fsub_rn(o[2 * j], f.x), __fsub_rn(o[2 * j + 1], f.y));
          }
          store_tile(stage, w, p.d_lo, p.ldd, row0, c0, p.m, p.n);
        }
      }
    }
    cur = next;
    __syncwarp();
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncwarp();
  return ok;
}

// The two issuing roles run with their whole warp, on values that are the
// same in every lane, and one elected lane issues: the operands of tensor-core
// and TMA instructions are then formed in uniform registers. From a branch
// that one lane takes alone, four MMAs and a commit took 370 clocks to issue
// and a load 410, more than a 128 x 64 stage needs.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool warp_wait(unsigned long long* bar, uint32_t parity,
                                          const int* failed) {
  return __all_sync(0xFFFFFFFFu, wait_parity_or_failed<false>(bar, parity, failed));
}

// The warp that loads one operand (A: 128 rows, B: BN) into the ring, tile
// after tile. A box holds 64 columns; K-major operands come as one box of all
// rows, MN-major ones as a box of 64 k rows for every 64 of the tile's rows.
template <int BN, bool A>
struct NsLoader {
  using L = NsLayout<BN>;
  static constexpr uint32_t kOp = A ? L::kA : L::kB;
  uint8_t* base;
  unsigned long long *full, *empty;
  int* failed;
  const bool lead;
  uint32_t n, s, ph;  // stages loaded so far, and where the next one goes
  __device__ NsLoader(uint8_t* sm, unsigned long long* full_, unsigned long long* empty_,
                      int* failed_, uint32_t loaded = 0)
      : base(A ? sm : sm + L::kBOff), full(full_), empty(empty_), failed(failed_),
        lead(elect_one()), n(loaded), s(loaded % L::kStages), ph((loaded / L::kStages) & 1u) {}
  __device__ __forceinline__ bool tile(const CUtensorMap* map, bool mn, int row0, int n_kb) {
    for (int kb = 0; kb < n_kb; ++kb) {
      if (!warp_wait(&empty[s], ph ^ 1u, failed)) {
        atomicExch(failed, 1);
        return false;
      }
      load(map, mn, row0, kb * kSK);
    }
    return __all_sync(0xFFFFFFFFu, !failed_flag(failed));
  }
  __device__ __forceinline__ void load(const CUtensorMap* map, bool mn, int row0, int k0) {
    uint8_t* const to = base + s * kOp;
    unsigned long long* const bar = &full[s];
    if (lead) {
      expect_tx(bar, kOp);
      if (mn) {
#pragma unroll
        for (int j = 0; j < int(kOp / 8192); ++j)
          tma_load_2d(to + j * 8192, map, row0 + 64 * j, k0, bar);
      } else {
        tma_load_2d(to, map, k0, row0, bar);
      }
    }
    if (++s == L::kStages) s = 0, ph ^= 1u;
    ++n;
  }
  // After a failure loads that no MMA waited for may be in flight, and one of
  // the two loading warps may have gone further than the other. That one loads
  // as many stages (their space was free when the other took it), so that
  // every phase begun completes, and waits for them.
  __device__ __forceinline__ void drain(const CUtensorMap* map, bool mn, const uint32_t* counts) {
    const uint32_t most = counts[0] > counts[1] ? counts[0] : counts[1];
    while (n < most) load(map, mn, 0, 0);
    for (uint32_t i = n < L::kStages ? 0 : n - L::kStages; i < n; ++i)
      wait_parity(&full[i % L::kStages], (i / L::kStages) & 1u);
    __syncwarp();
  }
};

// The warp that issues the MMAs, tile after tile into the two accumulators in
// turn.
template <int BN>
struct NsIssuer {
  using L = NsLayout<BN>;
  uint8_t* sm;
  unsigned long long *full, *empty;
  uint32_t tmem;
  int* failed;
  const bool lead;
  uint64_t a0, b0;
  uint32_t ka, kb_, idesc, s = 0, ph = 0, ti = 0;
  __device__ NsIssuer(uint8_t* sm_, unsigned long long* full_, unsigned long long* empty_,
                      uint32_t tmem_, int* failed_)
      : sm(sm_), full(full_), empty(empty_), tmem(tmem_), failed(failed_), lead(elect_one()) {}
  // majorness of the operands of the tiles that follow
  __device__ __forceinline__ void operands(bool a_mn, bool b_mn) {
    a0 = a_mn ? smem_desc_mn(sm) : smem_desc_sw128(sm);
    b0 = b_mn ? smem_desc_mn(sm + L::kBOff) : smem_desc_sw128(sm + L::kBOff);
    ka = a_mn ? 128u : 2u, kb_ = b_mn ? 128u : 2u;
    idesc = L::idesc(a_mn, b_mn);
  }
  __device__ __forceinline__ bool tile(int n_kb, unsigned long long* acc_full,
                                       unsigned long long* acc_empty) {
    const uint32_t buf = ti & 1, bph = (ti >> 1) & 1u;
    if (!warp_wait(&acc_empty[buf], bph ^ 1u, failed)) return false;
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t acc = tmem + buf * BN;
    bool ok = true;
    for (int kb = 0; kb < n_kb; ++kb) {
      if (!warp_wait(&full[s], ph, failed)) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;");
      const uint64_t ad = a0 + s * (L::kA >> 4), bd = b0 + s * (L::kB >> 4);
      unsigned long long* const bar = &empty[s];
      if (lead) {
#pragma unroll
        for (uint32_t j = 0; j < kSK / 16; ++j)
          mma_f16(acc, ad + j * ka, bd + j * kb_, idesc, (kb > 0 || j > 0) ? 1u : 0u);
        commit_to(bar);
      }
      if (++s == L::kStages) s = 0, ph ^= 1u;
    }
    if (lead) commit_to(&acc_full[buf]);
    __syncwarp();
    ++ti;
    return ok;
  }
  // every MMA issued has completed
  __device__ __forceinline__ void finish(bool ok, unsigned long long* drain) {
    if (!ok) atomicExch(failed, 1);
    if (lead) commit_to(drain);
    __syncwarp();
    if (!wait_parity(drain, 0)) atomicExch(failed, 1);
    __syncwarp();
  }
};

template <int BN, bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(kSThreads, 1)
    k_ns_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const NsArgs p) {
  using L = NsLayout<BN>;
  constexpr bool kSym = MODE == kGram || MODE == kSquare;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned long long* full = reinterpret_cast<unsigned long long*>(sm + L::kBarOff);
  unsigned long long* empty = full + L::kStages;
  unsigned long long* acc_full = empty + L::kStages;  // two accumulators
  unsigned long long* acc_empty = acc_full + 2;
  unsigned long long* drain = acc_empty + 2;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
  int* failed = reinterpret_cast<int*>(tmem_base + 1);
  uint32_t* counts = tmem_base + 2;  // stages that the two loading warps loaded
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int64_t mt = (p.m + kSM - 1) / kSM, nt = (p.n + BN - 1) / BN;
  const int64_t n_tiles = ns_tiles<BN>(kSym, mt, nt);
  const int n_kb = int((p.k + kSK - 1) / kSK);

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 2;" ::"r"(smem_u32(&full[s])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&empty[s])));
    }
    for (int s = 0; s < 2; ++s) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&acc_full[s])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&acc_empty[s])),
                   "r"(kSEpiWarps));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(drain)));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *failed = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_base)),
                 "r"(L::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  const uint32_t tmem = *tmem_base;
  // the next launch may set itself up now; this one reads what the launch
  // before it wrote, so every thread waits for that to have finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 0) {
    NsLoader<BN, true> ld(sm, full, empty, failed);
    for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x) {
      int64_t m0, n0;
      ns_tile<BN, kSym>(t, mt, nt, m0, n0);
      if (!ld.tile(&tm_a, A_MN, int(m0), n_kb)) break;
    }
    if (ld.lead) counts[0] = ld.n;
  } else if (warp == kSLoadB) {
    NsLoader<BN, false> ld(sm, full, empty, failed);
    for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x) {
      int64_t m0, n0;
      ns_tile<BN, kSym>(t, mt, nt, m0, n0);
      if (!ld.tile(&tm_b, B_MN, int(n0), n_kb)) break;
    }
    if (ld.lead) counts[1] = ld.n;
  } else if (warp == 1) {
    NsIssuer<BN> mma(sm, full, empty, tmem, failed);
    mma.operands(A_MN, B_MN);
    bool ok = true;
    for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x)
      ok = mma.tile(n_kb, acc_full, acc_empty);
    mma.finish(ok, drain);
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    int64_t ti = 0;
    for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x, ++ti) {
      int64_t m0, n0;
      ns_tile<BN, kSym>(t, mt, nt, m0, n0);
      const uint32_t buf = uint32_t(ti & 1), bph = uint32_t(ti >> 1) & 1u;
      const bool ok = ns_epilogue<BN, MODE, kSym>(p, m0 + 32 * q + lane, n0 + (BN / 2) * half,
                                            tmem + buf * BN + (uint32_t(32 * q) << 16) +
                                                uint32_t((BN / 2) * half),
                                            sm + L::kEpiOff + (warp - 2) * (32 * 80),
                                            &acc_full[buf], bph, failed);
      if (ok && lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&acc_empty[buf]))
                     : "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  report_failure(p.status, failed);
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(L::kTmemCols));
  // (last, where only the loading warps come by: before the two lines above it
  // cost each launch of 256 x 512 0.2 us)
  if (warp != 0 && warp != kSLoadB) return;
  if (__builtin_expect(failed_flag(failed), 0)) {
    if (warp == 0)
      NsLoader<BN, true>(sm, full, empty, failed, counts[0]).drain(&tm_a, A_MN, counts);
    else
      NsLoader<BN, false>(sm, full, empty, failed, counts[1]).drain(&tm_b, B_MN, counts);
  }
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles by pairs of CTAs (tcgen05 cta_group::2). With one CTA a tile
// of 128 x 256 an SM takes in 48 KB for 512 clocks of MMAs, more than its port
// to L2 delivers (64 bytes a clock): the loads alone took 3.1 of 4.0 ms on
// 4096 x 14336. In a pair each CTA loads its 128 rows of A and half of B's
// 256, 32 KB a stage, and the tensor cores of both read both halves. The CTA
// of rank 0 leads: it issues the MMAs for both, and the stages' barriers are
// its own; the loads of both CTAs complete on them, and its commits arrive in
// both CTAs.
// ---------------------------------------------------------------------------

struct PairLayout {
  static constexpr int kStages = 6;
  static constexpr uint32_t kA = kSM * 128, kB = kSM * 128;
  static constexpr uint32_t kBOff = kStages * kA;
  static constexpr uint32_t kEpiOff = kBOff + kStages * kB;
  static constexpr uint32_t kBarOff = kEpiOff + kSEpiWarps * 32 * 80;
  static constexpr uint32_t kBytes = kBarOff + 256;
  __host__ __device__ static constexpr uint32_t idesc(bool a_mn, bool b_mn) {
    return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(256 >> 3) << 17) | (uint32_t(256 >> 4) << 24);
  }
};

// The address of the same shared-memory byte in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A load into this CTA's shared memory that completes on the barrier at
// cluster address `bar`, which may be the other CTA's.
__device__ __forceinline__ void pair_load(void* dst, const CUtensorMap* map, int x, int y,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t tmem_c, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_c),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Arrive on the barrier at bar's offset in both CTAs once this thread's MMAs
// have completed.
__device__ __forceinline__ void pair_commit(unsigned long long* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"(uint16_t(3)));
}

template <bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(kSThreads, 1)
    k_ns_pair(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const NsArgs p) {
  using L = PairLayout;
  constexpr bool kSym = MODE == kGram || MODE == kSquare;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned long long* full = reinterpret_cast<unsigned long long*>(sm + L::kBarOff);
  unsigned long long* empty = full + L::kStages;
  unsigned long long* acc_full = empty + L::kStages;  // two accumulators
  unsigned long long* acc_empty = acc_full + 2;
  unsigned long long* drain = acc_empty + 2;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
  int* failed = reinterpret_cast<int*>(tmem_base + 1);
  uint32_t* counts = tmem_base + 2;  // stages that the two loading warps loaded
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t mt = (p.m + 255) / 256, nt = (p.n + 255) / 256;
  const int64_t n_tiles = kSym ? nt * (nt + 1) / 2 : mt * nt;
  const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
  const int n_kb = int((p.k + kSK - 1) / kSK);
  // rows of this CTA and columns of the pair
  auto tile_at = [&](int64_t t, int64_t& m0, int64_t& n0) {
    int64_t i, j;
    if constexpr (kSym) {
      // column j of the upper triangle has j + 1 tiles; the longest first
      for (j = nt - 1; t > j; --j) t -= j + 1;
      i = t;
    } else {
      constexpr int64_t G = 8;  // row tiles swept together (their panels stay in L2)
      const int64_t per = G * nt, g = t / per, r = t % per;
      const int64_t gm = mt - g * G < G ? mt - g * G : G;
      i = g * G + r % gm, j = r / gm;
    }
    m0 = i * 256 + int64_t(rank) * kSM, n0 = j * 256;
  };
  auto fail = [&] {
    // both CTAs of the pair give up together
    atomicExch(failed, 1);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(failed, rank ^ 1u)), "r"(1)
                 : "memory");
  };

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&full[s])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&empty[s])));
    }
    for (int s = 0; s < 2; ++s) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&acc_full[s])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&acc_empty[s])),
                   "r"(2 * kSEpiWarps));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(drain)));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *failed = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  pair_sync();  // barriers and tensor memory of both CTAs are ready
  asm volatile("tcgen05.fence::after_thread_sync;");
  const uint32_t tmem = *tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The loading warps (A's and B's of both CTAs). A's warp of the leading CTA
  // announces the whole stage: four loads of 16 KB (a load may complete before
  // that: the count goes below zero). `loaded`: stages so far.
  const bool loader = warp == 0 || warp == kSLoadB, is_a = warp == 0;
  const bool mn = is_a ? A_MN : B_MN;
  uint32_t s = 0, ph = 0, loaded = 0;
  auto load = [&](bool lead, int row0, int k0) {
    const CUtensorMap* const map = is_a ? &tm_a : &tm_b;
    uint8_t* const to = (is_a ? sm : sm + L::kBOff) + s * L::kA;
    const uint32_t bar = peer_addr(&full[s], 0);
    if (lead) {
      if (is_a && rank == 0) expect_tx(&full[s], 2 * (L::kA + L::kB));
      if (mn) {
        pair_load(to, map, row0, k0, bar);
        pair_load(to + 8192, map, row0 + 64, k0, bar);
      } else {
        pair_load(to, map, k0, row0, bar);
      }
    }
    if (++s == L::kStages) s = 0, ph ^= 1u;
    ++loaded;
  };
  if (loader) {
    const bool lead = elect_one();
    bool ok = true;
    for (int64_t t = first; t < n_tiles && ok; t += step) {
      int64_t m0, n0;
      tile_at(t, m0, n0);
      const int row0 = int(is_a ? m0 : n0 + int64_t(rank) * kSM);
      for (int kb = 0; kb < n_kb; ++kb) {
        if (!warp_wait(&empty[s], ph ^ 1u, failed)) {
          ok = false;
          break;
        }
        load(lead, row0, kb * kSK);
      }
      ok = ok && __all_sync(0xFFFFFFFFu, !failed_flag(failed));
    }
    if (!ok) fail();
    if (lead) counts[is_a ? 0 : 1] = loaded;
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const bool lead = elect_one();
      const uint64_t a0 = A_MN ? smem_desc_mn(sm) : smem_desc_sw128(sm);
      const uint64_t b0 = B_MN ? smem_desc_mn(sm + L::kBOff) : smem_desc_sw128(sm + L::kBOff);
      constexpr uint32_t ka = A_MN ? 128u : 2u, kb_ = B_MN ? 128u : 2u;
      uint32_t ti = 0;
      bool ok = true;
      for (int64_t t = first; t < n_tiles && ok; t += step, ++ti) {
        const uint32_t buf = ti & 1, bph = (ti >> 1) & 1u;
        if (!warp_wait(&acc_empty[buf], bph ^ 1u, failed)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;");
        const uint32_t acc = tmem + buf * 256;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!warp_wait(&full[s], ph, failed)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;");
          const uint64_t ad = a0 + s * (L::kA >> 4), bd = b0 + s * (L::kB >> 4);
          unsigned long long* const bar = &empty[s];
          if (lead) {
#pragma unroll
            for (uint32_t j = 0; j < kSK / 16; ++j)
              pair_mma(acc, ad + j * ka, bd + j * kb_, L::idesc(A_MN, B_MN),
                       (kb > 0 || j > 0) ? 1u : 0u);
            pair_commit(bar);
          }
          if (++s == L::kStages) s = 0, ph ^= 1u;
        }
        if (lead) pair_commit(&acc_full[buf]);
        __syncwarp();
      }
      if (!ok) fail();
      // every MMA issued has completed, and with them the loads that they read
      if (lead)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(drain)));
      __syncwarp();
      if (!wait_parity(drain, 0)) fail();
      __syncwarp();
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    int64_t ti = 0;
    for (int64_t t = first; t < n_tiles; t += step, ++ti) {
      int64_t m0, n0;
      tile_at(t, m0, n0);
      const uint32_t buf = uint32_t(ti & 1), bph = uint32_t(ti >> 1) & 1u;
      const bool ok = ns_epilogue<256, MODE, kSym>(
          p, m0 + 32 * q + lane, n0 + 128 * half,
          tmem + buf * 256 + (uint32_t(32 * q) << 16) + uint32_t(128 * half),
          sm + L::kEpiOff + (warp - 2) * (32 * 80), &acc_full[buf], bph, failed);
      if (lane == 0) {
        if (ok)
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                           peer_addr(&acc_empty[buf], 0))
                       : "memory");
        else
          fail();
      }
      __syncwarp();
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  pair_sync();  // neither CTA ends while the other's MMAs, loads or arrivals reach it
  if (failed_flag(failed)) {  // (in both CTAs or in neither)
    // The loading warps stopped at different stages, and loads that nobody
    // read may be in flight. All of them load as many stages as the furthest
    // did (whose space was free when that one took it), so that every phase
    // begun completes, and the leading CTA waits for these.
    if (loader) {
      uint32_t most = 0;
      for (uint32_t r = 0; r < 2; ++r) {
        for (uint32_t i = 0; i < 2; ++i) {
          uint32_t c;
          asm volatile("ld.shared::cluster.u32 %0, [%1];"
                       : "=r"(c)
                       : "r"(peer_addr(&counts[i], r))
                       : "memory");
          most = c > most ? c : most;
        }
      }
      const bool lead = elect_one();
      while (loaded < most) load(lead, 0, 0);
      if (is_a && rank == 0) {
        const uint32_t from = most < L::kStages ? 0 : most - L::kStages;
        for (uint32_t i = from; i < most; ++i)
          wait_parity(&full[i % L::kStages], (i / L::kStages) & 1u);
      }
      __syncwarp();
    }
    pair_sync();
  }
  report_failure(p.status, failed);
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// Sum of the squares of G in fp64: partial[b] over this CTA's elements.
template <bool BF16>
__device__ __forceinline__ float ns_load(const void* g, int64_t i) {
  return BF16 ? __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(g) + i)) << 16)
              : __ldg(static_cast<const float*>(g) + i);
}
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_ns_norm(const void* __restrict__ g, int64_t n, double* __restrict__ partial) {
  constexpr int VEC = BF16 ? 8 : 4;
  __shared__ double sh[8];
  double s = 0.0;
  const int64_t nv = n / VEC, stride = int64_t(gridDim.x) * 256;
  const int64_t me = int64_t(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t i = me; i < nv; i += stride) {
    const uint4 r = ld_stream(static_cast<const uint8_t*>(g) + 16 * i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        const double a = bf16_lo(w[j]), b = bf16_hi(w[j]);
        s += a * a + b * b;
      } else {
        const double a = __uint_as_float(w[j]);
        s += a * a;
      }
    }
  }
  for (int64_t i = nv * VEC + me; i < n; i += stride) {
    const double a = ns_load<BF16>(g, i);
    s += a * a;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) s += sh[i];
    partial[blockIdx.x] = s;
  }
}

// X = 2^12 G / (|G|_F + eps) as hi + lo, pitch ld. Every CTA adds the
// partial sums itself, in one order.
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_ns_start(const void* __restrict__ g, int64_t rows, int64_t cols, int64_t ld, float eps,
               const double* __restrict__ partial, int n_partial, __half* __restrict__ hi,
               __half* __restrict__ lo) {
  __shared__ float f[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += 32) s += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (threadIdx.x == 0) {
      // the factor as a power of two and a rest in [1, 2): G may be far from 1
      const double k = double(kNsScale) / (sqrt(s) + double(eps));
      int e = 0;
      if (k > 0.0 && k < 1e300) e = ilogb(k);
      e = e < -126 ? -126 : (e > 127 ? 127 : e);
      f[0] = exp2f(float(e));
      f[1] = float(scalbn(k, -e));
    }
  }
  __syncthreads();
  const float p = f[0], r = f[1];
  const int64_t chunks = (cols + 7) / 8;
  const bool vec = cols % 8 == 0;  // g is 16-byte aligned
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * chunks;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t row = i / chunks, c = i % chunks * 8;
    float v[8];
    if (vec) {
      if constexpr (BF16) {
        const uint4 q = ld_stream(static_cast<const uint16_t*>(g) + row * cols + c);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(w[j]), v[2 * j + 1] = bf16_hi(w[j]);
      } else {
        const float* at = static_cast<const float*>(g) + row * cols + c;
        const uint4 q0 = ld_l1(at), q1 = ld_l1(at + 4);
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = c + j < cols ? ns_load<BF16>(g, row * cols + c + j) : 0.0f;
    }
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = __fmul_rn(__fmul_rn(v[2 * j], p), r);
      const float b = __fmul_rn(__fmul_rn(v[2 * j + 1], p), r);
      hw[j] = pack_h2(a, b);
      const float2 h = unpack_h2(hw[j]);
      lw[j] = pack_h2(__fsub_rn(a, h.x), __fsub_rn(b, h.y));
    }
    *reinterpret_cast<uint4*>(hi + row * ld + c) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *reinterpret_cast<uint4*>(lo + row * ld + c) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
  }
}

// Tensor map over fp16 [rows][cols] with pitch ld: boxes of 64 columns (one
// 128-byte swizzle row) x box_rows.
bool encode_half(CUtensorMap* map, const __half* base, int64_t rows, int64_t cols, int64_t ld,
                 uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int ns_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <typename... P, typename... A>
cudaError_t ns_launch(void (*kern)(P...), int grid, int threads, size_t smem, cudaStream_t s,
                      A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// An fp16 matrix of the workspace and how a product reads it: K along its
// columns (K-major) or along its rows (MN-major).
struct NsOperand {
  const __half* p;
  int64_t rows, cols, ld;
  bool mn;
};

template <int BN, bool A_MN, bool B_MN, int MODE>
cudaError_t ns_gemm_bn(const NsOperand& a, const NsOperand& b, const NsArgs& args,
                       cudaStream_t s) {
  using L = NsLayout<BN>;
  CUtensorMap ta, tb;
  if (!encode_half(&ta, a.p, a.rows, a.cols, a.ld, A_MN ? kSK : kSM) ||
      !encode_half(&tb, b.p, b.rows, b.cols, b.ld, B_MN ? kSK : BN))
    return cudaErrorInvalidValue;
  auto kern = k_ns_gemm<BN, A_MN, B_MN, MODE>;
  constexpr size_t smem = L::kBytes + 1024;
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ns_tiles<BN>(MODE == kGram || MODE == kSquare, (args.m + kSM - 1) / kSM,
                                     (args.n + BN - 1) / BN);
  const int sms = ns_sms();
  return ns_launch(kern, int(tiles < sms ? tiles : sms), kSThreads, smem, s, ta, tb, args);
}

template <bool A_MN, bool B_MN, int MODE>
cudaError_t ns_gemm_pair(const NsOperand& a, const NsOperand& b, const NsArgs& args,
                         cudaStream_t s) {
  using L = PairLayout;
  CUtensorMap ta, tb;
  if (!encode_half(&ta, a.p, a.rows, a.cols, a.ld, A_MN ? kSK : kSM) ||
      !encode_half(&tb, b.p, b.rows, b.cols, b.ld, B_MN ? kSK : kSM))
    return cudaErrorInvalidValue;
  auto kern = k_ns_pair<A_MN, B_MN, MODE>;
  constexpr size_t smem = L::kBytes + 1024;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t mt = (args.m + 255) / 256, nt = (args.n + 255) / 256;
  const int64_t tiles = MODE == kGram || MODE == kSquare ? nt * (nt + 1) / 2 : mt * nt;
  const int64_t pairs = ns_sms() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, args);
}

// Tiles: 256 x 256 by pairs where there are two rounds of them or nearly
// (a round's epilogue then overlaps the next) and ragged edges leave little of
// them idle; else 128 columns where those fill two thirds of the GPU, else 64.
template <bool A_MN, bool B_MN, int MODE>
cudaError_t ns_gemm(const NsOperand& a, const NsOperand& b, const NsArgs& args, cudaStream_t s) {
  constexpr bool sym = MODE == kGram || MODE == kSquare;
  const int64_t mt = (args.m + kSM - 1) / kSM;
  const int64_t m2 = (args.m + 255) / 256, n2 = (args.n + 255) / 256;
  const int64_t pairs = 74, tiles = sym ? n2 * (n2 + 1) / 2 : m2 * n2;
  const int64_t rounds = (tiles + pairs - 1) / pairs;
  const double used = double(args.m) * double(args.n) / (sym ? 2 : 1);
  if (tiles >= kNsPairTiles && used >= 0.7 * double(rounds * pairs) * 65536.0)
    return ns_gemm_pair<A_MN, B_MN, MODE>(a, b, args, s);
  if (ns_tiles<128>(sym, mt, (args.n + 127) / 128) >= 100)
    return ns_gemm_bn<128, A_MN, B_MN, MODE>(a, b, args, s);
  return ns_gemm_bn<64, A_MN, B_MN, MODE>(a, b, args, s);
}

int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }
int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

int64_t newton_schulz_workspace(int64_t rows, int64_t cols) {
  const int64_t s = rows < cols ? rows : cols;
  return 3 * pad256(rows * pad64(cols) * 2) + 2 * pad256(s * pad64(s) * 2) + kNsPartials * 8;
}

cudaError_t launch_newton_schulz(const void* g, bool bf16, int64_t rows, int64_t cols, int steps,
                                 float a, float b, float c, float eps, float scale, void* out,
                                 bool out_bf16, void* workspace, int* status, cudaStream_t st) {
  const int64_t ldx = pad64(cols), s = rows < cols ? rows : cols, lds = pad64(s);
  const bool tall = rows > cols;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  const int64_t xb = pad256(rows * ldx * 2), sb = pad256(s * lds * 2);
  __half* x[2] = {reinterpret_cast<__half*>(w), reinterpret_cast<__half*>(w + xb)};
  __half* xl = reinterpret_cast<__half*>(w + 2 * xb);
  __half* ga = reinterpret_cast<__half*>(w + 3 * xb);
  __half* gb = reinterpret_cast<__half*>(w + 3 * xb + sb);
  double* partial = reinterpret_cast<double*>(w + 3 * xb + 2 * sb);

  const int64_t n = rows * cols;
  const int64_t want = (n / 8 + 255) / 256;
  const int n_partial = int(want < 1 ? 1 : (want < kNsPartials ? want : kNsPartials));
  if (bf16)
    k_ns_norm<true><<<n_partial, 256, 0, st>>>(g, n, partial);
  else
    k_ns_norm<false><<<n_partial, 256, 0, st>>>(g, n, partial);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t chunk_blocks = (rows * ((cols + 7) / 8) + 255) / 256;
  const int start_grid = int(chunk_blocks < 148 * 8 ? chunk_blocks : 148 * 8);
  e = bf16 ? ns_launch(k_ns_start<true>, start_grid, 256, 0, st, g, rows, cols, ldx, eps,
                       static_cast<const double*>(partial), n_partial, x[0], xl)
           : ns_launch(k_ns_start<false>, start_grid, 256, 0, st, g, rows, cols, ldx, eps,
                       static_cast<const double*>(partial), n_partial, x[0], xl);
  const NsOperand og = {ga, s, s, lds, false}, ob = {gb, s, s, lds, false};
  for (int i = 0; i < steps && e == cudaSuccess; ++i) {
    const __half* xi = x[i & 1];
    NsArgs p = {};
    p.status = status;
    // A = X X^T (X^T X): K along the longer side
    p.m = p.n = s, p.k = tall ? rows : cols;
    p.ldd = lds, p.alpha = kNsInv, p.d_hi = ga;
    NsOperand ox = {xi, rows, cols, ldx, tall};
    e = tall ? ns_gemm<true, true, kGram>(ox, ox, p, st) : ns_gemm<false, false, kGram>(ox, ox, p, st);
    if (e != cudaSuccess) break;
    // B = b A + c A A
    p.k = s, p.alpha = c * kNsInv, p.beta = b, p.c_hi = ga, p.d_hi = gb;
    e = ns_gemm<false, false, kSquare>(og, og, p, st);
    if (e != cudaSuccess) break;
    // X = a X + B X (a X + X B)
    p.m = rows, p.n = cols, p.k = s, p.ldd = ldx;
    p.alpha = kNsInv, p.beta = a, p.c_hi = xi, p.c_lo = xl, p.d_hi = x[(i + 1) & 1], p.d_lo = xl;
    p.out = out, p.out_bf16 = out_bf16, p.out_vec = cols % 8 == 0, p.out_scale = scale * kNsInv;
    ox.mn = !tall;
    if (i + 1 < steps)
      e = tall ? ns_gemm<false, false, kStep>(ox, ob, p, st) : ns_gemm<false, true, kStep>(ob, ox, p, st);
    else
      e = tall ? ns_gemm<false, false, kLast>(ox, ob, p, st) : ns_gemm<false, true, kLast>(ob, ox, p, st);
  }
  return e;
}

}  // namespace mxfp4
