// Products of a few bf16 rows with an MXFP4 weight (sm_100a):
//   Y[t][i] = sum_k X[t][k] W[i][k],  W[i][k] = G(code) 2^(scale byte - 127)
// with one scale per 32 elements along k. X is not quantized: this is the
// product a model answers with, where mxfp4_gemm's 4-bit activations would
// cost accuracy and where a step reads the whole weight for a few rows.
//
// Bound by reading the weight once (17/32 byte per element). The tensor cores
// take the weight as it lies in memory (kind::mxf4, packed codes, blocked
// scale tiles), so it never passes through a register; decoding on the CUDA
// cores costs about 1.5 instructions per weight, half of an SM's issue slots
// at full memory speed, before any arithmetic on x.
//
// X as an MXFP4 operand, without loss: every x of a group of 32 is written in
// balanced base-8 digits d_p, which are E2M1 values,
//   x = 2^s (d_0 + d_1 / 8 + ... + d_7 / 8^7) + rest,
// 2^s the power of two that puts the group's largest |x| into [2, 4): each
// digit is the nearest E2M1 value to what the digits before it left, at most
// 4 in magnitude, so it leaves at most 1/2, the next digit's 4. Digit p of
// all tokens is one block of rows of the B operand with group scales
// 2^(s - 3 p), and an accumulator column sums one digit of one token; the
// epilogue adds a token's 8 columns, the smallest first. x is exact where
// |x| is at least 2^-16 of its group's maximum, and otherwise off by at most
// 2^-23 of that maximum. With few rows the extra columns are free: reading
// the 128 weight rows of an MMA from shared memory takes it longer than 64
// columns of products. (Splitting x into two E4M3 values instead needs
// kind::mxf8f6f4, whose MMAs take 32 k instead of 64 and 16 bytes of shared
// memory for 8 of codes: the issue of its MMAs bound the kernel at 4.7 TB/s.)
//
// One CTA takes 128 weight rows, T tokens (N = 8 T columns) and a slab of k;
// the CTAs of a cluster take the slabs of the same rows and add their sums
// through distributed shared memory in the order of their ranks (no atomics).
//   warp 0:    one thread issues the loads of a stage (256 k: codes, scale
//              tiles, digits) into a ring;
//   warp 1:    tensor memory; one thread issues per stage the scale copies
//              and four MMAs (M = 128, N = 8 T, K = 64);
//   warps 2-5: for one or two tokens, write their digits into the stages
//              (every CTA for itself: one launch, no workspace); epilogue.
// For more tokens the digits cost more instructions than a stage leaves time
// for, so k_gemv_digits writes them once, in the order in which a stage reads
// them, and k_gemv is launched over it: it sets up and loads weights
// meanwhile and waits before it reads digits.
//
// Measured: 1 x 8192 x 28672 24.2 us (5.2 TB/s, 79% of a plain copy's rate),
// 1 x 4096 x 4096 6.5 us, 16 x 4096 x 14336 14.5 us. What is left is the
// start of a launch and the joining of slabs, about 5 us together. (MMAs that
// took turns on up to four accumulators were 2 to 9% slower than one.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include "launch.cuh"
#include "mxfp4_device.cuh"
#include "tc_common.cuh"

namespace mxfp4 {

namespace {

constexpr int kVM = 128;       // weight rows of a tile
constexpr int kVDigits = 8;    // digits of an x
constexpr int kVThreads = 192;
constexpr uint32_t kVNaN = 0x7FC00000u;

template <int T>
struct VLayout {
  static constexpr int kN = kVDigits * T;
  static constexpr int kRowBlocks = (kN + 127) / 128;      // scale tiles of B per 128 k
  static constexpr int kStages = T == 2 ? 5 : (T == 8 ? 4 : (T == 16 ? 3 : 4));
  static constexpr int kPerSm = T == 32 ? 1 : 2;           // CTAs an SM
  // bytes of a stage: codes, their scales, digits and their scales (the last
  // two as one block, the unit of the digit workspace)
  static constexpr uint32_t kA = kVM * 128, kSfa = 1024;
  static constexpr uint32_t kB = kN * 128, kSfb = 1024 * kRowBlocks;
  static constexpr uint32_t kX = kB + kSfb;
  static constexpr uint32_t kXOff = kStages * kA;
  static constexpr uint32_t kSfaOff = kXOff + kStages * kX;
  static constexpr uint32_t kPartOff = kSfaOff + kStages * kSfa;
  static constexpr uint32_t kBarOff = kPartOff + T * kVM * 4;
  static constexpr uint32_t kBytes = kBarOff + 256;
  static_assert(kPerSm * (kBytes + 2048) <= 227 * 1024, "CTAs an SM");
  static_assert(kX % 1024 == 0, "swizzle atoms");
  // tensor memory: accumulator, then per stage the scales of A (8 columns)
  // and B (8 a row block), so that copying a stage's scales waits for no MMA
  static constexpr uint32_t kSfCol = kN;
  static constexpr uint32_t kSfStage = 8 + 8 * kRowBlocks;
  static constexpr uint32_t kTmemUsed = kSfCol + kSfStage * kStages;
  static constexpr uint32_t kTmemCols = kTmemUsed <= 128 ? 128 : (kTmemUsed <= 256 ? 256 : 512);
  static_assert(kTmemCols * kPerSm <= 512 && kTmemUsed <= kTmemCols, "tensor memory");
  // kind::mxf4: E2M1 both (1), N / 8, E8M0 scales, M / 16
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (uint32_t(kN >> 3) << 17) |
                                     (1u << 23) | (uint32_t(kVM >> 4) << 24);
};

__device__ __forceinline__ void v_mma(uint32_t tmem_c, uint64_t adesc, uint64_t bdesc,
                                      uint32_t idesc, uint32_t accumulate, uint32_t tsfa,
                                      uint32_t tsfb) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, "
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

// The issuing warps run together on values that are the same in every lane,
// and one elected lane issues: the operands of tensor-core and TMA
// instructions are then formed in uniform registers (from a branch that one
// lane takes alone each of them takes 70 to 90 clocks to issue).
__device__ __forceinline__ bool v_elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool v_warp_wait(unsigned long long* bar, uint32_t parity,
                                            const int* failed) {
  return __all_sync(0xFFFFFFFFu, v_wait(bar, parity, failed));
}

__device__ __forceinline__ uint32_t v_cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void v_cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void v_cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void v_peer_store(uint32_t a, uint32_t rank, float v) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d), "f"(v) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
  if (BF16)
    static_cast<uint16_t*>(y)[at] = uint16_t(pack_bf16x2(v, 0.0f));
  else
    static_cast<float*>(y)[at] = v;
}

// Digits of 8 elements of a group that 4 adjacent lanes share, in packed
// codes: put(p, word, byte) for each digit p, byte its scale byte. A group
// with Inf or NaN gets scale byte 0xFF (NaN) for every digit.
template <typename Put>
__device__ __forceinline__ void digits8(uint4 raw, Put put) {
  uint32_t am = bf16x8_absmax(raw);
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  // byte of 2^s (s = exponent - 1, no lower than what digit 7 can reach)
  const bool bad = am >= 0x7F800000u;
  const uint32_t s0 = bad ? 0xFFu : max(am >> 23, 3u * (kVDigits - 1) + 1) - 1;
  const float mul = inv_scale(s0);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bad ? 0.0f : __fmul_rn(bf16_lo(w[j]), mul);
    v[2 * j + 1] = bad ? 0.0f : __fmul_rn(bf16_hi(w[j]), mul);
  }
#pragma unroll
  for (int p = 0; p < kVDigits; ++p) {
    put(p, e2m1x8_rn(v), bad ? 0xFFu : s0 - 3 * p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fsub_rn(v[j], e2m1_rn_value(v[j])), 8.0f);
  }
}

// A stage's B operand: row p T + t holds digit p of token t, 128 bytes of
// codes (256 k), 16-byte chunk c (a group) at c ^ (row % 8): the 128-byte
// swizzle; behind the kN rows the scale tiles [128-k half][row block].
template <int T>
__device__ __forceinline__ void put_digit(uint8_t* block, int p, int t, int g, int sub,
                                          uint32_t word, uint32_t byte) {
  using L = VLayout<T>;
  const int r = p * T + t;
  *reinterpret_cast<uint32_t*>(block + r * 128 + ((g ^ (r & 7)) << 4) + sub * 4) = word;
  if (sub == 0)
    block[L::kB + (g / 4 * L::kRowBlocks + r / 128) * 512 + 16 * (r % 32) + 4 * (r % 128 / 32) +
          g % 4] = uint8_t(byte);
}

// The digits of X: block tt * stages + kb holds the operand of token tile tt
// and stage kb. A thread takes 8 elements; groups from k on (up to whole MMAs
// of 64) get zeros.
template <int T>
__global__ void __launch_bounds__(256)
    k_gemv_digits(const uint16_t* __restrict__ x, int64_t ldx, int m, int64_t k, int64_t k64,
                  int stages, uint8_t* __restrict__ digits) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t per = k64 / 8;  // threads a token
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t token = id / per, e = (id - token * per) * 8;
  const bool in = token < m;    // whole groups: 4 threads agree
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (in && e < k) raw = ld_l1(x + token * ldx + e);
  uint8_t* const block =
      digits + ((token / T) * stages + e / 256) * int64_t(VLayout<T>::kX);
  digits8(raw, [&](int p, uint32_t word, uint32_t byte) {
    if (in)
      put_digit<T>(block, p, int(token % T), int(e % 256) / 32, int(e % 32) / 8, word, byte);
  });
}

struct VShape {
  int m, steps, stages, split;  // steps: MMAs of 64 k; stages: of 256
  int64_t n, k, k_tiles, ldx;   // k_tiles: scale tiles of 128 k
};

// OWN: the CTA writes the digits of x itself; else `digits` holds them.
template <int T, bool OWN, bool BF16>
__global__ void __launch_bounds__(kVThreads)
    k_gemv(const __grid_constant__ CUtensorMap tm_w, const uint8_t* __restrict__ sfw,
           const uint16_t* __restrict__ x, const uint8_t* __restrict__ digits, const VShape sh,
           void* __restrict__ y, int* __restrict__ status) {
  using L = VLayout<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned long long* full = reinterpret_cast<unsigned long long*>(sm + L::kBarOff);
  unsigned long long* empty = full + L::kStages;
  unsigned long long* acc_full = empty + L::kStages;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(acc_full + 1);
  int* failed = reinterpret_cast<int*>(tmem_base + 1);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int split = sh.split;
  const int rank = split > 1 ? int(v_cluster_rank()) : 0;
  const int64_t tile = blockIdx.x / split;
  const int64_t n0 = tile * kVM;
  const int t0 = int(blockIdx.y) * T;
  const int tokens = min(T, sh.m - t0);
  // this CTA's slab of stages
  const int kb0 = int(int64_t(sh.stages) * rank / split);
  const int kb1 = int(int64_t(sh.stages) * (rank + 1) / split);

  if (split > 1) v_cluster_arrive();  // waited for before the first store to a peer
  // the loads of a stage, by one thread
  auto load_w = [&](int kb, uint32_t s) {
    // (the last stage may have one scale tile)
    const uint32_t sf = 2 * kb + 1 < sh.k_tiles ? 1024u : 512u;
    expect_tx(&full[s], L::kA + sf + (OWN ? 0 : L::kX));
    tma_load_2d(sm + s * L::kA, &tm_w, kb * 128, int(n0), &full[s]);
    v_bulk_load(sm + L::kSfaOff + s * L::kSfa, sfw + (tile * sh.k_tiles + 2 * kb) * 512, sf,
                &full[s]);
  };
  auto load_x = [&](int kb, uint32_t s) {
    if (OWN) return;
    v_bulk_load(sm + L::kXOff + s * L::kX,
                digits + (int64_t(blockIdx.y) * sh.stages + kb) * int64_t(L::kX), L::kX,
                &full[s]);
  };
  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      // the loads' announcement, and each token's digits where written here
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[s])),
                   "r"(OWN ? 1 + tokens : 1));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&empty[s])));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(acc_full)));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    *failed = 0;
    // the first stages are free, and their weights need not wait for digits
    for (int i = 0; i < L::kStages && kb0 + i < kb1; ++i) load_w(kb0 + i, uint32_t(i));
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_base)),
                 "r"(L::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // OWN: item i of this CTA is token i % tokens of stage i / tokens; warp w
  // takes items w, w + active, ... (a lane 8 of the token's 256 elements) and
  // loads one ahead. Warps take turns over at most kStages stages: one that
  // is done with stage i knows that stage i - kStages has been consumed, and
  // the barrier of a later stage reads right only if the stage two rounds of
  // the ring before it has been consumed (phases alternate), so it must not
  // be more than kStages stages ahead of that. (Tokens that are absent leave
  // their rows as they are: an MMA column depends on its own row alone.)
  const int w = warp - 2;
  const int n_items = OWN ? (kb1 - kb0) * tokens : 0;
  const int active = OWN ? min(4, L::kStages * tokens) : 1;
  auto fetch = [&](int i) {
    const int st = i / tokens;
    const int64_t e = int64_t(kb0 + st) * 256 + 8 * lane;
    return i < n_items && e < sh.k ? ld_l1(x + (t0 + i - st * tokens) * sh.ldx + e)
                                   : make_uint4(0, 0, 0, 0);
  };
  uint4 next = make_uint4(0, 0, 0, 0);
  if (OWN && warp >= 2 && w < active) next = fetch(w);
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  const uint32_t tmem = *tmem_base;

  if (warp == 0) {
    const bool lead = v_elect();
    if (!OWN) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (lead)
        for (int i = 0; i < L::kStages && kb0 + i < kb1; ++i) load_x(kb0 + i, uint32_t(i));
    }
    // stages with a load, and the phase of each one's last
    uint32_t s = 0, ph = 1, issued = (1u << min(L::kStages, kb1 - kb0)) - 1, last_ph = 0;
    for (int kb = kb0 + L::kStages; kb < kb1; ++kb) {
      if (!v_warp_wait(&empty[s], ph ^ 1u, failed)) {
        atomicExch(failed, 1);
        break;
      }
      last_ph = (last_ph & ~(1u << s)) | (ph << s);
      if (lead) {
        load_w(kb, s);
        load_x(kb, s);
      }
      if (++s == L::kStages) s = 0, ph ^= 1u;
    }
    // every load has landed before the CTA can end
    for (uint32_t st = 0; st < L::kStages; ++st)
      if ((issued >> st) & 1u) v_wait(&full[st], (last_ph >> st) & 1u, nullptr);
    __syncwarp();
  } else if (warp == 1) {
    const bool lead = v_elect();
    const uint64_t a0 = smem_desc_sw128(sm), x0 = smem_desc_sw128(sm + L::kXOff);
    const uint64_t fa0 = smem_desc(sm + L::kSfaOff, 16, 128);
    const uint64_t fb0 = smem_desc(sm + L::kXOff + L::kB, 16, 128);
    const uint32_t sf0 = tmem + L::kSfCol;
    bool ok = true;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1 && ok; kb += L::kStages, ph ^= 1u) {
#pragma unroll
      for (int s = 0; s < L::kStages; ++s) {
        if (kb + s >= kb1) break;
        if (!v_warp_wait(&full[s], ph, failed)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;");
        const int left = sh.steps - 4 * (kb + s);  // MMAs of this stage, up to 4
        const uint32_t sfa = sf0 + L::kSfStage * s, sfb = sfa + 8;
        if (lead) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (2 * j >= left) break;
            v_copy_desc(sfa + 4 * j, fa0 + (s * L::kSfa + j * 512) / 16);
#pragma unroll
            for (int h = 0; h < L::kRowBlocks; ++h)
              v_copy_desc(sfb + 4 * (j * L::kRowBlocks + h),
                          fb0 + (s * L::kX + (j * L::kRowBlocks + h) * 512) / 16);
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (g >= left) break;
            const uint32_t id = 2u * (g & 1);
            v_mma(tmem, a0 + (s * (L::kA >> 4) + 2 * g),
                  x0 + (s * (L::kX >> 4) + 2 * g), L::kIdesc | (id << 29) | (id << 4),
                  (s > 0 || g > 0 || kb > kb0) ? 1u : 0u,
                  (sfa + 4 * (g >> 1)) | (id << 30),
                  (sfb + 4 * (g >> 1) * L::kRowBlocks) | (id << 30));
          }
          commit_to(&empty[s]);
        }
      }
    }
    if (!ok) atomicExch(failed, 1);
    if (lead) commit_to(acc_full);
    __syncwarp();
    // the MMAs issued have completed before shared or tensor memory goes
    if (!v_wait(acc_full, 0, nullptr)) atomicExch(failed, 1);
    __syncwarp();
  } else if (OWN) {
    for (int i = w < active ? w : n_items; i < n_items; i += active) {
      const int st = i / tokens, t = i - st * tokens;
      const uint32_t s = uint32_t(st % L::kStages), ph = uint32_t(st / L::kStages) & 1u;
      const uint4 raw = next;
      next = fetch(i + active);
      if (!__all_sync(0xFFFFFFFFu, v_wait(&empty[s], ph ^ 1u, failed))) {
        atomicExch(failed, 1);
        break;
      }
      uint8_t* const block = sm + L::kXOff + s * L::kX;
      digits8(raw, [&](int p, uint32_t word, uint32_t byte) {
        put_digit<T>(block, p, t, lane >> 2, lane & 3, word, byte);
      });
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&full[s]))
                     : "memory");
    }
  }
  // Epilogue: warp w reads lane quarter w % 4, rows 32 q + lane. In a cluster
  // the rows are shared out for the joining, 128 / split to a rank: every
  // rank stores its sums for them at their owner, which adds them in order.
  const int share = kVM / split;      // split is a power of two
  if (split > 1) v_cluster_wait();    // every CTA of the cluster has started
  if (warp >= 2) {
    const bool bad = !v_wait(acc_full, 0, failed,
                             kAccWaitLimit < kVWaitLimit ? kAccWaitLimit : kVWaitLimit) ||
                     failed_flag(failed);
    if (bad) atomicExch(failed, 1);
    const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
    asm volatile("tcgen05.fence::after_thread_sync;");
    const int q = warp & 3, row = 32 * q + lane;
    const uint32_t tb = tmem + (uint32_t(32 * q) << 16);
    const int owner = row / share;
    const uint32_t part = smem_u32(sm + L::kPartOff);
    constexpr int kC = T < 4 ? T : 4;  // tokens a round
#pragma unroll 1
    for (int c = 0; c < tokens; c += kC) {
      float v[kC];
      uint32_t r[kVDigits][4];
#pragma unroll
      for (int p = 0; p < kVDigits; ++p) {
        const uint32_t at = tb + p * T + c;
        if constexpr (kC == 2)
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
                       : "=r"(r[p][0]), "=r"(r[p][1])
                       : "r"(at));
        else
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(r[p][0]), "=r"(r[p][1]), "=r"(r[p][2]), "=r"(r[p][3])
                       : "r"(at));
      }
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        v[j] = __uint_as_float(r[kVDigits - 1][j]);
#pragma unroll
        for (int p = kVDigits - 2; p >= 0; --p) v[j] = __fadd_rn(v[j], __uint_as_float(r[p][j]));
      }
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const int t = c + j;
        if (t >= tokens) break;
        if (any_bad) v[j] = __uint_as_float(kVNaN);
        if (split > 1)  // [rank][token][row of the share]
          v_peer_store(part + 4 * ((rank * T + t) * share + row - owner * share),
                       uint32_t(owner), v[j]);
        else if (n0 + row < sh.n)
          store_y<BF16>(y, int64_t(t0 + t) * sh.n + n0 + row, v[j]);
      }
      __syncwarp();
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
  }
  if (split > 1) {
    __syncwarp();
    v_cluster_arrive();
    v_cluster_wait();
    const float* part = reinterpret_cast<const float*>(sm + L::kPartOff);
    for (int i = tid; i < tokens * share; i += kVThreads) {
      const int t = i / share, r = i % share;
      float v = part[t * share + r];
      for (int k = 1; k < split; ++k) v = __fadd_rn(v, part[(k * T + t) * share + r]);
      const int64_t row = n0 + rank * share + r;
      if (row < sh.n) store_y<BF16>(y, int64_t(t0 + t) * sh.n + row, v);
    }
  }
  __syncthreads();
  report_failure(status, failed);
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(L::kTmemCols));
}

struct GemvArgs {
  const uint16_t* x;
  int64_t m, n, k, ldx;
  const uint8_t *codes, *scales;
  void* y;
  uint8_t* digits;
  int* status;
  cudaStream_t s;
};

int gemv_tokens(int64_t m) { return m <= 2 ? 2 : (m <= 8 ? 8 : (m <= 16 ? 16 : 32)); }

// Slabs of k (a power of two up to the portable cluster size): up to one CTA
// an SM in any case, up to `per_sm` CTAs an SM (whose loads together keep an
// SM's share of the memory bandwidth busy) where that leaves a slab four
// stages. 8192 x 28672 (2 CTAs an SM / 1): 23.8 / 24.6 us; 4096 x 4096, with
// slabs of 2 / 4 stages: 8.3 / 6.5 us (clusters start one after another).
int gemv_split(int64_t tiles, int64_t stages, int per_sm) {
  int split = 1;
  while (split < 8 && stages >= 2 * split &&
         (tiles * split * 2 <= 148 ||
          (tiles * split * 2 <= 148 * per_sm && stages >= 8 * split)))
    split *= 2;
  return split;
}

template <int T, bool BF16>
cudaError_t gemv_t(const GemvArgs& a) {
  using L = VLayout<T>;
  constexpr bool kOwn = T == 2;
  VShape sh;
  sh.m = int(a.m);
  sh.steps = int((a.k + 63) / 64);
  sh.stages = int((a.k + 255) / 256);
  sh.n = a.n;
  sh.k = a.k;
  sh.k_tiles = (a.k + 127) / 128;
  sh.ldx = a.ldx;
  const int64_t tiles = (a.n + kVM - 1) / kVM, t_tiles = (a.m + T - 1) / T;
  sh.split = gemv_split(tiles * t_tiles, sh.stages, L::kPerSm);

  CUtensorMap tm;
  if (!encode_rows_sw128(&tm, a.codes, a.n, a.k / 2, kVM)) return cudaErrorInvalidValue;
  auto kern = k_gemv<T, kOwn, BF16>;
  constexpr size_t smem = L::kBytes + 1024;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  if (!kOwn) {
    const int64_t k64 = int64_t(sh.steps) * 64, threads = a.m * (k64 / 8);
    k_gemv_digits<T><<<unsigned((threads + 255) / 256), 256, 0, a.s>>>(
        a.x, a.ldx, int(a.m), a.k, k64, sh.stages, a.digits);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles * sh.split), unsigned(t_tiles));
  cfg.blockDim = dim3(kVThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(sh.split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = kOwn ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kern, tm, a.scales, a.x,
                            static_cast<const uint8_t*>(a.digits), sh, a.y, a.status);
}

template <bool BF16>
cudaError_t gemv_any(const GemvArgs& a) {
  switch (gemv_tokens(a.m)) {
    case 2: return gemv_t<2, BF16>(a);
    case 8: return gemv_t<8, BF16>(a);
    case 16: return gemv_t<16, BF16>(a);
    default: return gemv_t<32, BF16>(a);
  }
}

}  // namespace

int64_t gemv_workspace(int64_t m, int64_t, int64_t k) {
  const int T = gemv_tokens(m);
  if (T == 2) return 0;
  const int64_t block =
      T == 8 ? VLayout<8>::kX : (T == 16 ? VLayout<16>::kX : VLayout<32>::kX);
  return (m + T - 1) / T * ((k + 255) / 256) * block;
}

cudaError_t launch_gemv(const void* x, int64_t m, int64_t n, int64_t k, int64_t ldx,
                        const uint8_t* codes, const uint8_t* scales, void* y, bool bf16_out,
                        void* workspace, int* status, cudaStream_t s) {
  const GemvArgs a = {static_cast<const uint16_t*>(x), m, n, k, ldx, codes, scales, y,
                      static_cast<uint8_t*>(workspace), status, s};
  return bf16_out ? gemv_any<true>(a) : gemv_any<false>(a);
}

}  // namespace mxfp4
