// Products of a few bf16 rows with an MXFP4 weight (sm_100a):
//   Y[t][i] = sum_k X[t][k] W[i][k],  W[i][k] = G(code) 2^(scale byte - 127)
// with one scale per 32 elements along k. X is not quantized: this is the
// product a model answers with, where mxfp4_gemm's 4-bit activations would
// cost accuracy and where a step reads the whole weight for a few rows.
//
// Bound by reading the weight once (17/32 byte per element). The tensor cores
// take E2M1 operands directly, so the weight goes from memory to them without
// passing through a register: a tensor-memory-access (TMA) load spreads each
// 16 packed codes over 16 bytes of shared memory (the operand layout of
// kind::mxf8f6f4), the blocked scale tile is copied to tensor memory, and one
// thread issues the MMAs. Decoding on the CUDA cores instead costs about 1.5
// instructions per weight, 2 issue slots per clock and SM of the 4 there are
// at full memory speed, before any arithmetic on x.
//
// X as an MMA operand: every bf16 x is split into two E4M3 values with a
// power-of-two scale per 32 elements of each,
//   hi = e4m3(x 2^-s),  lo = e4m3((x - hi 2^s) 2^-s'),
// s from the group's largest |x| and s' from its largest remainder. hi keeps
// 4 of bf16's 8 significant bits and lo the other 4, so the split is exact
// unless |x| is below 2^-13 of its group's maximum, and off by at most 2^-21
// of that maximum then (the products are summed in fp32). hi and lo are two
// rows of the B operand, their products two accumulator columns that the
// epilogue adds.
//
// Work: a tile is 128 weight rows x T tokens (N = 2 T columns), a unit 128 k
// of it. The units of all tiles, k first, are dealt out in equal runs to two
// CTAs an SM, so a run can end inside a tile: a tile that one run covers is
// stored at once, the sums of the others go to the caller's workspace and a
// second small kernel (launched ahead, waiting on the first) adds them in the
// order of k. No atomics: the same bits every time. (Clusters that joined
// their sums through distributed shared memory took 1.5 to 3 us to start: the
// clusters of a GPC start one after another.)
//   warp 0:    one thread issues the loads of codes (128 rows x 128 k) and
//              scale tiles into a ring of stages;
//   warp 1:    tensor memory; one thread issues per stage the two scale
//              copies and four MMAs (M = 128, N = 2 T, K = 32);
//   warps 2-:  split X into the stages, and where a run leaves a tile, read
//              the accumulators and store the sums.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "launch.cuh"
#include "mxfp4_device.cuh"
#include "tc_common.cuh"

namespace mxfp4 {

namespace {

constexpr int kVM = 128;                 // weight rows of a tile
constexpr int kVCtas = 296;              // runs: two CTAs an SM of a B200
constexpr uint32_t kVNaN = 0x7FC00000u;

template <int T>
struct VLayout {
  static constexpr int kN = 2 * T;
  // a warp splits 8 tokens at a time
  static constexpr int kWorkers = T == 8 ? 4 : 8;
  static constexpr int kThreads = 32 * (2 + kWorkers);
  // as many as let two CTAs share an SM
  static constexpr int kStages = T == 8 ? 5 : (T == 16 ? 5 : (T == 32 ? 4 : 3));
  // Accumulators: consecutive MMAs on one wait for each other's result, which
  // with few columns takes longer than the MMA itself, so the four K = 32
  // steps of a stage go to accumulators of their own where they fit.
  static constexpr int kAcc = T <= 16 ? 4 : (T == 32 ? 2 : 1);
  static constexpr uint32_t kA = kVM * 128, kB = kN * 128, kSf = 512;
  // per ring: codes, x planes, scales of both
  static constexpr uint32_t kAOff = 0;
  static constexpr uint32_t kBOff = kAOff + kStages * kA;
  static constexpr uint32_t kSfaOff = kBOff + kStages * kB;
  static constexpr uint32_t kSfbOff = kSfaOff + kStages * kSf;
  static constexpr uint32_t kBarOff = kSfbOff + kStages * kSf;
  static constexpr uint32_t kBytes = kBarOff + 256;
  static_assert(2 * (kBytes + 2048) <= 227 * 1024, "two CTAs an SM");
  // tensor memory: accumulators, then per stage 4 columns of either scales
  // (their own, so that copying a stage's scales waits for no MMA)
  static constexpr uint32_t kSfCol = kAcc * kN;
  static constexpr uint32_t kTmemUsed = kSfCol + 8 * kStages;
  static constexpr uint32_t kTmemCols = kTmemUsed <= 128 ? 128 : 256;
  static_assert(kTmemUsed <= 256, "two CTAs share an SM's 512 columns");
  // kind::mxf8f6f4: A E2M1 (5), B E4M3 (0), both K-major, N / 8, E8M0
  // scales, M / 16
  static constexpr uint32_t kIdesc =
      (5u << 7) | (0u << 10) | (uint32_t(kN >> 3) << 17) | (1u << 23) | (uint32_t(kVM >> 4) << 24);
};

__device__ __forceinline__ void mma_mxf8f6f4(uint32_t tmem_c, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate, uint32_t tsfa,
                                             uint32_t tsfb) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, "
      "%3, [%5], [%6], p;\n\t}\n" ::"r"(tmem_c),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(tsfa), "r"(tsfb));
}

// A 512-byte scale tile from shared memory (descriptor d) to 4 columns.
__device__ __forceinline__ void v_copy_desc(uint32_t taddr, uint64_t d) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d));
}

__device__ __forceinline__ void v_bulk_load(void* dst, const void* src, uint32_t bytes,
                                            unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
      "%2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// wait_parity_or_failed with a lower limit (these kernels run for
// microseconds): gives up as soon as another role of the CTA has.
constexpr long long kVWaitLimit = 1ll << 20;
__device__ __forceinline__ bool v_wait(unsigned long long* bar, uint32_t parity,
                                       const int* failed, long long limit = kVWaitLimit) {
  const uint32_t a = smem_u32(bar);
  for (long long i = 0; i < limit; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(a), "r"(parity)
        : "memory");
    if (done) return true;
    if (failed != nullptr && (i & 63) == 63 && failed_flag(failed)) return false;
  }
  return false;
}

// E4M3 code pairs (nearest, saturating at 448) of two fp32 values, and back.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void e4m3x2_decode(uint32_t c, float* out) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(h)
      : "r"(c));
  asm("{\n\t.reg .f16 l, u;\n\t"
      "mov.b32 {l, u}, %2;\n\t"
      "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(out[0]), "=f"(out[1])
      : "r"(h));
}

// Scale byte that puts a maximum of the given fp32 bit pattern into
// [128, 256) (smaller where the byte stops at 0); 0xFF for Inf and NaN.
__device__ __forceinline__ uint32_t plane_scale(uint32_t amax_bits) {
  const uint32_t E = amax_bits >> 23;
  return amax_bits >= 0x7F800000u ? 0xFFu : (E > 7u ? E - 7u : 0u);
}

// Both planes of 8 values of a group that 4 adjacent lanes share, for R
// independent groups at once (the shuffles and conversions of one hide behind
// those of the others: one at a time took 4 times as long).
struct Planes {
  uint2 hi, lo;
  uint32_t s_hi, s_lo;
};
template <int R>
__device__ __forceinline__ void split8(const uint4* raw, Planes* p) {
  uint32_t am[R], rm[R];
  float r[R][8];
#pragma unroll
  for (int k = 0; k < R; ++k) am[k] = bf16x8_absmax(raw[k]);
#pragma unroll
  for (int o = 1; o <= 2; o *= 2)
#pragma unroll
    for (int k = 0; k < R; ++k) am[k] = max(am[k], __shfl_xor_sync(0xFFFFFFFFu, am[k], o));
#pragma unroll
  for (int k = 0; k < R; ++k) {
    p[k].s_hi = plane_scale(am[k]);
    const bool bad = p[k].s_hi == 0xFFu;
    const float mul = inv_scale(p[k].s_hi);
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    uint32_t c[4];
    rm[k] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = __fmul_rn(bf16_lo(w[j]), mul), b = __fmul_rn(bf16_hi(w[j]), mul);
      c[j] = e4m3x2(a, b);
      float d[2];
      e4m3x2_decode(c[j], d);
      r[k][2 * j] = __fsub_rn(a, d[0]);  // exact: in units of 2^s_hi
      r[k][2 * j + 1] = __fsub_rn(b, d[1]);
      rm[k] = max(rm[k], max(__float_as_uint(r[k][2 * j]) & 0x7FFFFFFFu,
                             __float_as_uint(r[k][2 * j + 1]) & 0x7FFFFFFFu));
    }
    p[k].hi = bad ? make_uint2(0, 0) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    if (bad) rm[k] = 0;
  }
#pragma unroll
  for (int o = 1; o <= 2; o *= 2)
#pragma unroll
    for (int k = 0; k < R; ++k) rm[k] = max(rm[k], __shfl_xor_sync(0xFFFFFFFFu, rm[k], o));
#pragma unroll
  for (int k = 0; k < R; ++k) {
    // the remainders are at most 8 (half a step of 4 significant bits); the
    // remainders get a scale of their own, relative to s_hi and never below
    // 2^-127 (remainders below 2^-113 of s_hi, far under fp32's reach, shrink)
    const bool bad = p[k].s_hi == 0xFFu;
    int rel = rm[k] == 0 ? 0 : max(int(rm[k] >> 23) - 127 - 7, -120);
    if (int(p[k].s_hi) + rel < 0) rel = -int(p[k].s_hi);
    p[k].s_lo = bad ? 0u : uint32_t(int(p[k].s_hi) + rel);
    const float mul = __uint_as_float(uint32_t(127 - rel) << 23);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = e4m3x2(__fmul_rn(r[k][2 * j], mul), __fmul_rn(r[k][2 * j + 1], mul));
    p[k].lo = bad ? make_uint2(0, 0) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
}

template <bool BF16>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
  if (BF16)
    static_cast<uint16_t*>(y)[at] = uint16_t(pack_bf16x2(v, 0.0f));
  else
    static_cast<float*>(y)[at] = v;
}

// The shape of one call. Tile t covers weight rows 128 (t / t_tiles) and tokens
// T (t % t_tiles) on (token tiles of one weight tile run close together, so
// they find its codes in L2).
struct VShape {
  int m, kblocks, t_tiles, run;  // run: units of a CTA
  int64_t n, ldx, units;
};

template <int T, bool BF16>
__global__ void __launch_bounds__(VLayout<T>::kThreads, 2)
    k_gemv(const __grid_constant__ CUtensorMap tm_w, const uint8_t* __restrict__ sfw,
           const uint16_t* __restrict__ x, const VShape sh, void* __restrict__ y,
           float* __restrict__ partial, int* __restrict__ status) {
  using L = VLayout<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned long long* full = reinterpret_cast<unsigned long long*>(sm + L::kBarOff);
  unsigned long long* empty = full + L::kStages;
  unsigned long long* acc_full = empty + L::kStages;
  unsigned long long* acc_empty = acc_full + 1;
  unsigned long long* drain = acc_full + 2;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(acc_full + 3);
  int* failed = reinterpret_cast<int*>(tmem_base + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kblocks = sh.kblocks;
  // this CTA's run of units: `blocks` of them from k block kb_first of tile0
  const int64_t u0 = int64_t(blockIdx.x) * sh.run;
  const int blocks = int(sh.units - u0 < sh.run ? sh.units - u0 : sh.run);
  const int64_t tile0 = u0 / kblocks;
  const int kb_first = int(u0 - tile0 * kblocks);
  // split batches of a stage: the same number for every tile of the call
  const int n_batch = (min(sh.m, T) + 7) / 8;

  uint32_t issued = 0, last_ph = 0;  // loading thread: stages, last phases
  int l_kb = kb_first;               // ... and its next unit
  int64_t l_tile = tile0;
  auto load = [&](uint32_t s, uint32_t ph) {
    issued |= 1u << s;
    last_ph = (last_ph & ~(1u << s)) | (ph << s);
    const int64_t nt = sh.t_tiles == 1 ? l_tile : l_tile / sh.t_tiles;
    // the tile load counts the packed codes: half of the bytes it fills
    expect_tx(&full[s], L::kA / 2 + L::kSf);
    tma_load_2d(sm + L::kAOff + s * L::kA, &tm_w, l_kb * 128, int(nt * kVM), &full[s]);
    v_bulk_load(sm + L::kSfaOff + s * L::kSf, sfw + (nt * kblocks + l_kb) * 512, L::kSf,
                &full[s]);
    if (++l_kb == kblocks) l_kb = 0, ++l_tile;
  };
  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      // the loads' announcement and a split batch each
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[s])),
                   "r"(1 + n_batch));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&empty[s])));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(acc_full)));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(acc_empty)),
                 "r"(L::kWorkers));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(drain)));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    *failed = 0;
    // the first stages are free: their loads need not wait for the others
    for (int i = 0; i < blocks && i < L::kStages; ++i) load(uint32_t(i), 0);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_base)),
                 "r"(L::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  // Workers: X is split in batches of 8 tokens x 128 k (a lane holds 8
  // elements of a token, 16 lanes a token, two tokens a round), n_batch to a
  // stage. Warp w takes batches w, w + active, ... of the CTA's sequence and
  // loads two of its batches ahead. Warps take turns over at most kStages
  // stages: one that is done with block i knows that block i - kStages has
  // been consumed, and the barrier of a later block's stage reads right only
  // if the block two rounds of the ring before it has been consumed (phases
  // alternate), so it must not be more than kStages blocks ahead of that.
  // The planes of tokens that a tile lacks hold whatever was there: an MMA
  // column depends on its own row of the operand alone, and theirs are not
  // stored.
  const int w = warp - 2, half = lane >> 4, l16 = lane & 15;
  const int n_items = blocks * n_batch;
  const int active = min(L::kWorkers, L::kStages * n_batch);
  // unit of item i: its tile relative to tile0, k block and token base
  auto locate = [&](int i, int& blk, int& b, int& rel, int& kb, int& t0) {
    blk = n_batch == 1 ? i : i / n_batch;
    b = i - blk * n_batch;
    rel = (kb_first + blk) / kblocks;
    kb = kb_first + blk - rel * kblocks;
    t0 = sh.t_tiles == 1 ? 0 : int((tile0 + rel) % sh.t_tiles) * T;
  };
  int f_i = w < active ? w : n_items;  // the next batch to fetch
  struct Batch {
    uint4 r[4];
  };
  auto fetch = [&](Batch& q) {
    if (f_i < n_items) {
      int blk, b, rel, kb, t0;
      locate(f_i, blk, b, rel, kb, t0);
      const uint16_t* xp = x + int64_t(kb) * 128 + l16 * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + 8 * b + 2 * j + half;
        if (t < sh.m && 8 * b < T) q.r[j] = ld_l1(xp + int64_t(t) * sh.ldx);
      }
    }
    f_i += active;
  };
  Batch b0, b1, b2;
  if (warp >= 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) b0.r[j] = b1.r[j] = b2.r[j] = make_uint4(0, 0, 0, 0);
    fetch(b0);
    fetch(b1);
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  const uint32_t tmem = *tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 1;
      for (int i = L::kStages; i < blocks; ++i) {
        if (!v_wait(&empty[s], ph ^ 1u, failed)) {
          atomicExch(failed, 1);
          break;
        }
        load(s, ph);
        if (++s == L::kStages) s = 0, ph ^= 1u;
      }
      // every load has landed before the CTA can end (the workers' arrival
      // completes the phase too; after a failure the wait is only bounded)
      for (uint32_t st = 0; st < L::kStages; ++st)
        if ((issued >> st) & 1u) v_wait(&full[st], (last_ph >> st) & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // Issuing is what bounds this thread (about 70 ns a stage beside the
      // MMAs where addresses are formed in the loop): the loop is unrolled
      // over the ring, so that every operand is a base plus a constant.
      const uint64_t a0 = smem_desc_sw128(sm + L::kAOff), b0d = smem_desc_sw128(sm + L::kBOff);
      const uint64_t fa0 = smem_desc(sm + L::kSfaOff, 16, 128);
      const uint64_t fb0 = smem_desc(sm + L::kSfbOff, 16, 128);
      const uint32_t sf0 = tmem + L::kSfCol;
      bool ok = true;
      uint32_t ph = 0, seg = 0;
      int kb = kb_first;
      uint32_t fresh = 1;  // the next MMAs start their accumulators
      for (int i = 0; i < blocks && ok; i += L::kStages, ph ^= 1u) {
#pragma unroll
        for (int s = 0; s < L::kStages; ++s) {
          if (i + s >= blocks) break;
          // a new tile: its accumulators have been read
          if ((fresh && seg > 0 && !v_wait(acc_empty, (seg - 1) & 1u, failed)) ||
              !v_wait(&full[s], ph, failed)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;");
          const uint32_t sfa = sf0 + 8 * s, sfb = sfa + 4;
          v_copy_desc(sfa, fa0 + s * (L::kSf >> 4));
          v_copy_desc(sfb, fb0 + s * (L::kSf >> 4));
#pragma unroll
          for (uint32_t g = 0; g < 4; ++g)
            mma_mxf8f6f4(tmem + (g % L::kAcc) * L::kN, a0 + (s * (L::kA >> 4) + 2 * g),
                         b0d + (s * (L::kB >> 4) + 2 * g), L::kIdesc | (g << 29) | (g << 4),
                         g >= L::kAcc ? 1u : fresh ^ 1u, sfa + (g << 30), sfb + (g << 30));
          commit_to(&empty[s]);
          fresh = 0;
          if (++kb == kblocks || i + s + 1 == blocks) {
            commit_to(acc_full);
            ++seg;
            fresh = 1;
            kb = 0;
          }
        }
      }
      if (!ok) atomicExch(failed, 1);
      // the MMAs issued have completed before shared or tensor memory goes
      commit_to(drain);
      if (!v_wait(drain, 0, nullptr)) atomicExch(failed, 1);
    }
    __syncwarp();
  } else {
    const int segs = (kb_first + blocks + kblocks - 1) / kblocks;
    int i = w < active ? w : n_items;
    for (int seg = 0; seg < segs; ++seg) {
      // the batches of this tile
      for (; i < n_items; i += active) {
        int blk, b, rel, kb, t0;
        locate(i, blk, b, rel, kb, t0);
        if (rel != seg) break;
        const uint32_t s = uint32_t(blk % L::kStages), ph = uint32_t(blk / L::kStages) & 1u;
        fetch(b2);
        if (!__all_sync(0xFFFFFFFFu, v_wait(&empty[s], ph ^ 1u, failed))) {
          atomicExch(failed, 1);
          break;
        }
        uint8_t* const bt = sm + L::kBOff + s * L::kB;
        uint8_t* const ft = sm + L::kSfbOff + s * L::kSf + (l16 >> 2);
        auto put = [&](const Planes& p, int t) {
          // row r of the 128-byte swizzled K-major operand: 16-byte chunk c
          // at c ^ (r % 8); this lane's 8 codes are half a chunk
          const uint32_t c = uint32_t(l16 >> 1), o = uint32_t(l16 & 1) * 8;
          const uint32_t rl = uint32_t(T + t);
          *reinterpret_cast<uint2*>(bt + t * 128 + ((c ^ (t & 7)) << 4) + o) = p.hi;
          *reinterpret_cast<uint2*>(bt + rl * 128 + ((c ^ (rl & 7)) << 4) + o) = p.lo;
          if ((lane & 3) == 0) {
            ft[16 * (t & 31) + 4 * (t >> 5)] = uint8_t(p.s_hi);
            ft[16 * (rl & 31) + 4 * (rl >> 5)] = uint8_t(p.s_lo);
          }
        };
        if (sh.m - t0 - 8 * b <= 2) {
          Planes p[1];
          split8<1>(b0.r, p);
          put(p[0], 8 * b + half);
        } else {
          Planes p[4];
          split8<4>(b0.r, p);
#pragma unroll
          for (int j = 0; j < 4; ++j) put(p[j], 8 * b + 2 * j + half);
        }
        b0 = b1;
        b1 = b2;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&full[s]))
                       : "memory");
      }
      // the tile's sums: lane quarter q of tensor memory holds rows 32 q +
      // lane; with 8 workers two warps a quarter, half of the tokens each
      const int64_t tile = tile0 + seg;
      const int64_t nt = sh.t_tiles == 1 ? tile : tile / sh.t_tiles;
      const int t0 = int(tile - nt * sh.t_tiles) * T;
      const int tokens = min(T, sh.m - t0);
      const bool whole = (seg > 0 || kb_first == 0) && (seg + 1) * kblocks <= kb_first + blocks;
      const bool got = __all_sync(
          0xFFFFFFFFu, !failed_flag(failed) && v_wait(acc_full, uint32_t(seg) & 1u, failed,
                                                      kAccWaitLimit < kVWaitLimit ? kAccWaitLimit
                                                                                  : kVWaitLimit));
      if (!got) atomicExch(failed, 1);
      asm volatile("tcgen05.fence::after_thread_sync;");
      constexpr int kSpan = T * 4 / L::kWorkers;  // tokens of a warp
      const int q = warp & 3, row = 32 * q + lane, h = w >> 2;
      const uint32_t tb = tmem + (uint32_t(32 * q) << 16);
      float* const part = partial + (int64_t(blockIdx.x) + tile) * (T * kVM) + row;
#pragma unroll
      for (int c = h * kSpan; c < (h + 1) * kSpan; c += 4) {
        uint32_t a[L::kAcc][2][4];
#pragma unroll
        for (int k = 0; k < L::kAcc; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(a[k][e][0]), "=r"(a[k][e][1]), "=r"(a[k][e][2]), "=r"(a[k][e][3])
                         : "r"(tb + k * L::kN + e * T + c));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = 0.0f;
#pragma unroll
          for (int k = 0; k < L::kAcc; ++k)
            v = __fadd_rn(v, __fadd_rn(__uint_as_float(a[k][0][j]), __uint_as_float(a[k][1][j])));
          if (!got) v = __uint_as_float(kVNaN);
          if (c + j >= tokens) continue;
          if (!whole)
            part[(c + j) * kVM] = v;
          else if (nt * kVM + row < sh.n)
            store_y<BF16>(y, int64_t(t0 + c + j) * sh.n + nt * kVM + row, v);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;");
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(acc_empty))
                     : "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  report_failure(status, failed);
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(L::kTmemCols));
}

// Tiles that several runs share: run i's sums of tile t are at i + t (runs
// and tiles only ever go up together, so no two pairs share a place).
template <int T, bool BF16>
__global__ void __launch_bounds__(256)
    k_gemv_join(const float* __restrict__ partial, const VShape sh, void* __restrict__ y) {
  constexpr int kPer = T * kVM / 256;  // CTAs a tile
  const int64_t tile = blockIdx.x / kPer;
  const int e = int(blockIdx.x % kPer) * 256 + threadIdx.x;
  const int64_t first = tile * sh.kblocks / sh.run;
  const int64_t last = ((tile + 1) * sh.kblocks - 1) / sh.run;
  const int64_t nt = tile / sh.t_tiles;
  const int64_t t = (tile - nt * sh.t_tiles) * T + e / kVM, row = nt * kVM + e % kVM;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (first == last || t >= sh.m || row >= sh.n) return;
  const float* p = partial + (first + tile) * (T * kVM) + e;
  float v = __ldcg(p);
  int64_t i = first + 1;
  for (; i + 3 <= last; i += 4) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = __ldcg(p += T * kVM);
#pragma unroll
    for (int k = 0; k < 4; ++k) v = __fadd_rn(v, q[k]);
  }
  for (; i <= last; ++i) v = __fadd_rn(v, __ldcg(p += T * kVM));
  store_y<BF16>(y, t * sh.n + row, v);
}

// Any k that is a multiple of 32 (the tensor-core kernel takes multiples of
// 128) and codes that are not 32-byte aligned: a warp takes a weight row, a
// lane a group of 32 (16 bytes of codes) at a time, for TB tokens.
template <int TB, bool BF16>
__global__ void __launch_bounds__(256)
    k_gemv_simt(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf,
                const uint16_t* __restrict__ x, int64_t ldx, int m, int64_t n, int64_t k,
                void* __restrict__ y) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t0 = int(blockIdx.y) * TB;
  if (row >= n) return;
  const int64_t groups = k / 32, k_tiles = (groups + 3) / 4;
  const uint8_t* c = codes + row * (k / 2);
  const uint8_t* f = sf + (row / 128) * k_tiles * 512 + 16 * (row % 32) + 4 * (row % 128 / 32);
  float acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.0f;
  for (int64_t g = lane; g < groups; g += 32) {
    const uint4 cw = ld_stream(c + 16 * g);
    const uint32_t sb = __ldg(f + (g >> 2) * 512 + (g & 3));
    const float scale = sb == 0xFFu ? __uint_as_float(kVNaN) : scale_value(sb);
    const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
    float sum[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) sum[t] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float wv[8];
      e2m1x8_decode(w[j], wv);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int tt = min(t0 + t, m - 1);
        const uint4 xv = ld_l1(x + int64_t(tt) * ldx + g * 32 + 8 * j);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[t] = __fmaf_rn(wv[2 * i], bf16_lo(xw[i]), sum[t]);
          sum[t] = __fmaf_rn(wv[2 * i + 1], bf16_hi(xw[i]), sum[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[t] = __fmaf_rn(sum[t], scale, acc[t]);
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      acc[t] = __fadd_rn(acc[t], __shfl_xor_sync(0xFFFFFFFFu, acc[t], o));
    if (lane == t && t0 + t < m) store_y<BF16>(y, int64_t(t0 + t) * n + row, acc[t]);
  }
}

// Tensor map of the codes [n][k / 2]: boxes of 128 elements x 128 rows, each
// 16 codes spread over 16 bytes of shared memory, 128-byte swizzle.
bool encode_codes(CUtensorMap* map, const void* codes, int64_t n, int64_t k) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cuuint64_t(k), cuuint64_t(n)};
  const cuuint64_t strides[1] = {cuuint64_t(k / 2)};
  const cuuint32_t box[2] = {128, uint32_t(kVM)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(codes), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct GemvArgs {
  const uint16_t* x;
  int64_t m, n, k, ldx;
  const uint8_t *codes, *scales;
  void* y;
  void* workspace;
  int* status;
  cudaStream_t s;
};

int gemv_tokens(int64_t m) { return m <= 8 ? 8 : (m <= 16 ? 16 : (m <= 32 ? 32 : 64)); }

// How the units are dealt out. Runs of at least two units; runs that hold
// several tiles anyway are rounded up to whole tiles, which saves the joining
// (about 2 us) for at most a quarter more work in the longest run.
VShape gemv_shape(int64_t m, int64_t n, int64_t k, int64_t ldx) {
  const int T = gemv_tokens(m);
  VShape sh;
  sh.m = int(m);
  sh.kblocks = int(k / 128);
  sh.t_tiles = int((m + T - 1) / T);
  sh.n = n;
  sh.ldx = ldx;
  sh.units = (n + kVM - 1) / kVM * sh.t_tiles * sh.kblocks;
  int64_t run = (sh.units + kVCtas - 1) / kVCtas;
  if (run < 2) run = 2;
  if (run >= 4 * int64_t(sh.kblocks) || sh.kblocks == 1)
    run = (run + sh.kblocks - 1) / sh.kblocks * sh.kblocks;
  sh.run = int(run);
  return sh;
}

template <int T, bool BF16>
cudaError_t gemv_tc(const GemvArgs& a) {
  using L = VLayout<T>;
  CUtensorMap tm;
  if (!encode_codes(&tm, a.codes, a.n, a.k)) return cudaErrorInvalidValue;
  auto kern = k_gemv<T, BF16>;
  constexpr size_t smem = L::kBytes + 1024;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const VShape sh = gemv_shape(a.m, a.n, a.k, a.ldx);
  const unsigned grid = unsigned((sh.units + sh.run - 1) / sh.run);
  float* partial = static_cast<float*>(a.workspace);
  kern<<<grid, L::kThreads, smem, a.s>>>(tm, a.scales, a.x, sh, a.y, partial, a.status);
  e = cudaGetLastError();
  if (e != cudaSuccess || sh.run % sh.kblocks == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sh.units / sh.kblocks * (T * kVM / 256)));
  cfg.blockDim = dim3(256);
  cfg.stream = a.s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_gemv_join<T, BF16>, static_cast<const float*>(partial), sh,
                            a.y);
}

template <bool BF16>
cudaError_t gemv_any(const GemvArgs& a) {
  if (a.k % 128 == 0 && (reinterpret_cast<uintptr_t>(a.codes) & 31u) == 0) {
    switch (gemv_tokens(a.m)) {
      case 8: return gemv_tc<8, BF16>(a);
      case 16: return gemv_tc<16, BF16>(a);
      case 32: return gemv_tc<32, BF16>(a);
      default: return gemv_tc<64, BF16>(a);
    }
  }
  const dim3 grid(unsigned((a.n + 7) / 8), unsigned(a.m == 1 ? 1 : (a.m + 7) / 8));
  if (a.m == 1)
    k_gemv_simt<1, BF16><<<grid, 256, 0, a.s>>>(a.codes, a.scales, a.x, a.ldx, int(a.m), a.n, a.k,
                                                a.y);
  else
    k_gemv_simt<8, BF16><<<grid, 256, 0, a.s>>>(a.codes, a.scales, a.x, a.ldx, int(a.m), a.n, a.k,
                                                a.y);
  return cudaGetLastError();
}

}  // namespace

int64_t gemv_workspace(int64_t m, int64_t n, int64_t k) {
  if (k % 128 != 0) return 0;
  const VShape sh = gemv_shape(m, n, k, k);
  if (sh.run % sh.kblocks == 0) return 0;
  const int64_t runs = (sh.units + sh.run - 1) / sh.run;
  return (runs + sh.units / sh.kblocks) * gemv_tokens(m) * kVM * int64_t(sizeof(float));
}

cudaError_t launch_gemv(const void* x, int64_t m, int64_t n, int64_t k, int64_t ldx,
                        const uint8_t* codes, const uint8_t* scales, void* y, bool bf16_out,
                        void* workspace, int* status, cudaStream_t s) {
  const GemvArgs a = {static_cast<const uint16_t*>(x), m, n, k, ldx, codes, scales, y, workspace,
                      status, s};
  return bf16_out ? gemv_any<true>(a) : gemv_any<false>(a);
}

}  // namespace mxfp4
