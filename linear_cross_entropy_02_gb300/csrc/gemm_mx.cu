// out = cap(m A W^T) of microscaled 4-bit operands on the tensor cores:
// tcgen05.mma kind::mxf4 with a power-of-two scale per 32 elements, products
// summed in fp32 in tensor memory.
//
// Two kernels: up to 128 tokens, where W is streamed once and HBM bounds the time,
// and for more of them pairs of CTAs on 256 x 256 tiles (further down), bound by the
// tensor cores. In the first, W's rows are the M dimension (128 vocabulary entries
// per tile) and the tokens the N dimension (16 to 128): a lane of tensor memory is a
// vocabulary entry, and a warp's store for one token is one contiguous run of logits
// whatever the row stride's alignment. One token on 129280 x 7168 takes 79 us, 93% of
// the copy bandwidth; 128 on 128256 x 4096 take 57.
//
// K advances 256 elements (one 128-byte swizzle row of codes) per stage. Scales
// come from HBM already in the order of tensor memory, 512 bytes per 128 rows x
// 128 elements, by one bulk copy per stage and operand. Four warps of their own
// carry them on to tensor memory (every lane quarter needs a copy: each warp
// writes its own). tcgen05.cp would do that in one instruction, but it waits for
// the MMAs before it and they for it: with it a stage took 1080 cycles for one
// token as for 192, and one token on 129280 x 7168 took 111 us instead of 83.
// An instruction covers K = 64 and picks its two scale bytes of each column by
// the scale ids in its descriptor.
//
// For a few tokens A stays in shared memory, all of its K with its scales, if it
// leaves room for the ring: re-reading it for every tile of W cost 10 us of 82.
// Up to kMostFused elements are encoded by every CTA for itself, straight into
// the swizzled tiles, while the first copies of W are on their way: a launch less.
//
// Warp 0 loads, warp 1 issues the MMAs, warps 2-5 store, warps 6-9 carry scales;
// there are two accumulators, so that the stores of one tile run under the MMAs of the
// next. Every wait is bounded (flce_device.cuh) and ends the call with
// FLCE_ERR_TIMEOUT.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "flce_device.cuh"
#include "flce_host.h"
#include "head_device.cuh"
#include "head_internal.h"
#include "microscale_device.cuh"

namespace flce {

namespace {

constexpr int kTileV = 128;                // vocabulary rows per tile
constexpr int kStageK = 256;               // elements of K per stage
constexpr int kRowBytes = 128;             // bytes of a row per stage
constexpr int kWBytes = kTileV * kRowBytes;
constexpr int kSfTiles = kStageK / kMxTileCols;  // scale tiles per 128 rows and stage
constexpr int kThreads = 320;
constexpr int kSmemBudget = 226 * 1024;
// (Microseconds of a single cold call so, and with a launch before it: 5 tokens of 7168 on 129280
// entries 100.4 and 102.4, 8 102.4 and 102.6, 12 105.3 and 103.3; 8 of 4096 on 128256
// 66.7 and 69.9, 12 67.6 and 70.1, 16 70.0 and 70.2, 24 71.7 and 68; 37 of 1056 on 50257
// 20.5 and 23.6, 64 24.6 and 23.6; 16 of 2048 on 32000 18.4 and 21.5, 32 22.5 and 21.5.
// They meet between 50000 and 65000 elements on all four.)
constexpr int64_t kMostFused = 40960;

// Shared and tensor memory of a tile of NT tokens. RESIDENT: A's codes and scales
// stay in shared memory in front of the ring, which then holds W alone.
template <int NT, bool RESIDENT>
struct Plan {
  static constexpr int x_bytes = NT * kRowBytes;
  static constexpr int w_sf = kSfTiles * kMxTileBytes;
  static constexpr int x_sf = kSfTiles * kMxTileBytes;
  static constexpr int x_all = x_bytes + x_sf;  // of one stage's K
  static constexpr int stage = kWBytes + w_sf + (RESIDENT ? 0 : x_all);
  static constexpr int d_cols = NT < 32 ? 32 : NT;      // one accumulator
  static constexpr int sf_cols = 2 * 4 * kSfTiles;
  static constexpr int by_tmem = (512 - 2 * d_cols) / sf_cols;
  static constexpr int most = by_tmem < 10 ? by_tmem : 10;
  // Stages of the ring when k_iters stages' worth of A is resident (0: they do not fit).
  static constexpr int stages(int k_iters) {
    const int room = kSmemBudget - 2048 - (RESIDENT ? k_iters * x_all : 0);
    const int n = room / stage;
    return n > most ? most : n < 4 ? 0 : n;
  }
  static constexpr int smem(int k_iters) {
    return stages(k_iters) * stage + (RESIDENT ? k_iters * x_all : 0) + 1024 + 512;
  }
  static constexpr int used_cols = 2 * d_cols + most * sf_cols;
  static constexpr int tmem_cols = used_cols <= 128 ? 128 : used_cols <= 256 ? 256 : 512;
  static_assert(x_bytes % 1024 == 0, "operand tiles start on a swizzle atom");
};

struct MxArgs {
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  int rows, vocab, k_iters, k_tiles, k_mmas;  // k_mmas: instructions over all of K
  const void* x;  // FUSED: the tokens as they are
  int x_f32, cols;
  int64_t ld_x;
  int v_tiles, stages;
  float out_mult, softcap, inv_softcap;
  void* out;
  int64_t ld_out;
  int32_t* status;
  uint64_t timeout_ns;
  int stall;  // test hook: the MMA warp issues nothing, so that every other wait runs out
};

// Instruction descriptor of kind::mxf4: E2M1 operands (1 in bits 7-9 and 10-12),
// N >> 3 in bits 17-22, E8M0 scales (bit 23), M >> 4 in bits 24-28, and the
// scale ids of B (bits 4-5) and A (bits 29-30): the byte of each 32-bit column
// at which the instruction's two scales begin.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf) {
  return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// This lane's rows of two scale tiles (16 bytes each, in shared memory) into
// eight columns of this warp's lane quarter.
__device__ __forceinline__ void store_scales2(uint32_t tmem, const uint8_t* a, const uint8_t* b) {
  const uint4 u = *reinterpret_cast<const uint4*>(a), v = *reinterpret_cast<const uint4*>(b);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(tmem), "r"(u.x),
               "r"(u.y), "r"(u.z), "r"(u.w), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void store_scales_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of a converged warp. Loader and MMA warps run their loops as
// whole warps and issue from the elected lane: in code that a single lane runs,
// the compiler has to move every operand of an MMA or copy to uniform registers
// anew, and a stage of four MMAs took 1000 cycles instead of 400.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// For a thread of a CTA in which a wait gave up, after all of the CTA's warps have
// left their loops: copies may still be in flight, and the shared memory that they
// write to stays as long as this thread does. They land in microseconds.
constexpr uint64_t kDrainNs = 10 * 1000 * 1000;
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = global_timer_ns();
  for (int i = 0; i < 100000 && global_timer_ns() - t0 < kDrainNs; ++i) __nanosleep(1000);
}

// wait_bounded by a whole warp, which then agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, w));
}

// A sum of the accumulator as the logit that leaves the kernel.
__device__ __forceinline__ float finish(const MxArgs& p, uint32_t sum) {
  const float z = __uint_as_float(sum) * p.out_mult;
  return p.softcap > 0.f ? p.softcap * tanhf(z * p.inv_softcap) : z;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The tokens' codes and scales by warps 2 to 9, at the places that TMA with
// 128-byte swizzle would give them (16-byte piece c of a row is at c ^ (row & 7))
// and in the order of a scale tile. The last instruction's K is filled up with
// zeros; rows beyond the tokens are left as they are: their results are not stored.
template <int NT, typename T>
__device__ __forceinline__ void encode_tokens(const MxArgs& p, uint8_t* s_x, uint8_t* s_xsf) {
  using P = Plan<NT, true>;
  constexpr int kLanes = kThreads - 64;
  const int per_row = p.k_mmas * (64 / kUnit), real = p.cols / kUnit, total = p.rows * per_row;
  const bool wide = reinterpret_cast<uintptr_t>(p.x) % 32 == 0 && p.ld_x * sizeof(T) % 32 == 0;
  constexpr int kAhead = 4;  // units per lane whose loads are in flight together
  for (int base = 0; base < total; base += kAhead * kLanes) {
    uint32_t raw[kAhead][4 * sizeof(T)];
    int row[kAhead], u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = base + k * kLanes + threadIdx.x - 64;
      row[k] = i / per_row;
      u[k] = i < total ? i - row[k] * per_row : -1;
      if (u[k] >= 0 && u[k] < real) load16<T>(static_cast<const T*>(p.x) + row[k] * p.ld_x + u[k] * kUnit, wide, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool in = u[k] >= 0 && u[k] < real;
      uint32_t E = in ? exponent16(raw[k]) : 0;
      E = max(E, __shfl_xor_sync(0xffffffffu, E, 1));  // the other half of the block
      if (u[k] >= 0) {
        const int slice = u[k] / 16, piece = u[k] % 16 / 2;
        uint8_t* to = s_x + slice * P::x_bytes + row[k] * kRowBytes + ((piece ^ (row[k] & 7)) << 4) + (u[k] & 1) * 8;
        *reinterpret_cast<uint2*>(to) = in ? encode16(raw[k], E) : make_uint2(0u, 0u);
        if ((u[k] & 1) == 0)
          s_xsf[u[k] / 8 * kMxTileBytes + row[k] % 32 * 16 + row[k] / 32 * 4 + (u[k] / 2 & 3)] =
              static_cast<uint8_t>(in ? scale_byte(E) : 127u);
      }
    }
  }
}

template <int NT, bool RESIDENT, bool FUSED, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const MxArgs p) {
  static_assert(RESIDENT || !FUSED, "encoded tokens stay in shared memory");
  using P = Plan<NT, RESIDENT>;
  const int S = p.stages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int x_slots = RESIDENT ? p.k_iters : S;  // A's slices: all of them, or one per stage
  uint8_t* s_w = smem;
  uint8_t* s_x = s_w + S * kWBytes;
  uint8_t* s_wsf = s_x + x_slots * P::x_bytes;
  uint8_t* s_xsf = s_wsf + S * P::w_sf;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_xsf + x_slots * P::x_sf);
  uint64_t* empty = full + S;
  uint64_t* scaled = empty + S;  // the stage's scales are in tensor memory
  uint64_t* tfull = scaled + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint64_t* x_full = mma_done + 1;  // RESIDENT: all of A has arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(x_full + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // (the first wait can run out seconds after this, and all CTAs run at once)
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&scaled[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 128);
    }
    mbar_init(mma_done, 1);
    mbar_init(x_full, FUSED ? 8 : 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, P::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  if (FUSED && warp >= 2) {
    if (p.x_f32)
      encode_tokens<NT, float>(p, s_x, s_xsf);
    else
      encode_tokens<NT, uint16_t>(p, s_x, s_xsf);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(x_full);
  }

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool aborted = false;
    if (RESIDENT && !FUSED && elect_one()) {  // one tile of tokens, whose scales are one row of tiles
      mbar_arrive_expect_tx(x_full, p.k_iters * P::x_bytes + p.k_tiles * kMxTileBytes);
      for (int k = 0; k < p.k_iters; ++k) tma_load_2d(s_x + k * P::x_bytes, &map_x, x_full, k * kRowBytes, 0);
      bulk_load(s_xsf, p.x_scales, static_cast<uint32_t>(p.k_tiles) * kMxTileBytes, x_full);
    }
    __syncwarp();
    for (int vb = blockIdx.x; vb < p.v_tiles && !aborted; vb += gridDim.x) {
      for (int k = 0; k < p.k_iters; ++k) {
        if (!warp_wait(&empty[stage], phase ^ 1u, wc)) {
          aborted = true;
          break;
        }
        if (elect_one()) {
          const int kt = k * kSfTiles;
          const uint32_t sf = static_cast<uint32_t>(min(kSfTiles, p.k_tiles - kt)) * kMxTileBytes;
          mbar_arrive_expect_tx(&full[stage], kWBytes + sf + (RESIDENT ? 0 : P::x_bytes + sf));
          tma_load_2d(s_w + stage * kWBytes, &map_w, &full[stage], k * kRowBytes, vb * kTileV);
          bulk_load(s_wsf + stage * P::w_sf, p.w_scales + (static_cast<int64_t>(vb) * p.k_tiles + kt) * kMxTileBytes,
                    sf, &full[stage]);
          if (!RESIDENT) {
            tma_load_2d(s_x + stage * P::x_bytes, &map_x, &full[stage], k * kRowBytes, 0);
            bulk_load(s_xsf + stage * P::x_sf, p.x_scales + kt * kMxTileBytes, sf, &full[stage]);
          }
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    const uint32_t w0 = smem_u32(s_w), x0 = smem_u32(s_x);
    bool aborted = RESIDENT && !warp_wait(x_full, 0, wc);
    for (int vb = p.stall ? p.v_tiles : blockIdx.x; vb < p.v_tiles && !aborted; vb += gridDim.x) {
      if (!warp_wait(&tempty[acc], acc_phase ^ 1u, wc)) break;
      tc_fence_after_sync();
      const uint32_t d = tmem + static_cast<uint32_t>(acc * P::d_cols);
      for (int k = 0; k < p.k_iters; ++k) {
        if (!warp_wait(&full[stage], phase, wc) || !warp_wait(&scaled[stage], phase, wc)) {
          aborted = true;
          break;
        }
        tc_fence_after_sync();
        if (elect_one()) {
          const uint32_t sf = tmem + static_cast<uint32_t>(2 * P::d_cols + stage * P::sf_cols);
          const uint32_t sfx = sf + 4 * kSfTiles;
          const uint32_t a0 = w0 + stage * kWBytes, b0 = x0 + (RESIDENT ? k : stage) * P::x_bytes;
          const int mmas = p.k_mmas - k * (kStageK / 64);
#pragma unroll
          for (int j = 0; j < kStageK / 64; ++j)
            if (j < mmas)
              mma_mxf4(d, sdesc_kmajor_sw128(a0 + j * 32), sdesc_kmajor_sw128(b0 + j * 32),
                       idesc_mxf4(kTileV, NT, (j & 1) * 2), sf + 4 * (j >> 1), sfx + 4 * (j >> 1),
                       (k | j) != 0 ? 1u : 0u);
          tc_commit(&empty[stage]);
          if (k == p.k_iters - 1) tc_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (elect_one()) {
      tc_commit(mma_done);
      wait_drain(mma_done, 0, p.timeout_ns, p.status);
    }
    __syncwarp();
  } else if (warp >= 6) {
    // Scales of a stage whose copies have landed: its last MMAs are done, since the
    // loader waited for them, so its columns are free.
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = !RESIDENT || wait_bounded(x_full, 0, wc);
    for (int vb = blockIdx.x; vb < p.v_tiles && __all_sync(0xffffffffu, ok); vb += gridDim.x) {
      for (int k = 0; k < p.k_iters; ++k) {
        ok = wait_bounded(&full[stage], phase, wc);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after_sync();
        const uint32_t sf = t_lane + static_cast<uint32_t>(2 * P::d_cols + stage * P::sf_cols);
        const uint8_t* w = s_wsf + stage * P::w_sf + lane * 16;
        // (a last stage of one tile carries the stage before's bytes in the other's place: not used)
        store_scales2(sf, w, w + kMxTileBytes);
        const uint8_t* x = s_xsf + (RESIDENT ? k : stage) * P::x_sf + lane * 16;
        store_scales2(sf + 8, x, x + kMxTileBytes);
        store_scales_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&scaled[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int vb = blockIdx.x; vb < p.v_tiles; vb += gridDim.x) {
      const bool ok = wait_bounded(&tfull[acc], acc_phase, wc);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after_sync();
      const int v = vb * kTileV + quarter * 32 + lane;
      for (int c = 0; c < p.rows; c += 32) {
        uint32_t r[32];
        tmem_load_32cols(t_lane + acc * P::d_cols + c, r);
        tmem_load_wait_regs(r);
        T* o = static_cast<T*>(p.out) + static_cast<int64_t>(c) * p.ld_out + v;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (c + j < p.rows && v < p.vocab) o[j * p.ld_out] = from_float<T>(finish(p, r[j]));
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, P::tmem_cols);
  }
  if (threadIdx.x == 0 && *abort_flag) let_copies_land();
}

// More than 128 tokens: 256 x 256 tiles over a cluster of two CTAs on two SMs.
// A single CTA's 128 x 192 tile drew 43 KB per K = 256 for 384 cycles of MMAs, more
// than an SM gets from the L2: 4096 tokens on 128256 x 4096 took 1106 us, 786 of
// them with the MMAs left out. Here each CTA holds 128 rows of M and 128 of N, 35 KB
// with the scales for 512 cycles, and the same product takes 625 to 640 us (6.7 to
// 6.9 PFLOP/s) of encoded tokens in calls now and then, 700 (6.2) after hundreds back
// to back, when the clock falls; the MMAs alone 505, the copies alone 376. M = 256, N = 256 fill half of tensor
// memory, so that the other half holds scales and the accumulator is one: sixteen
// warps take it into registers at once and store from there, under the next tile's
// MMAs. Between two tiles the MMAs rest for about 960 of 8200 cycles.
//
// TOKENS_M: the tokens are M, a thread has 128 neighbouring logits of one token
// and stores whole 32-byte sectors, for which rows of logits start on 32 bytes.
// Else the vocabulary is M, and a warp's store is 32 neighbouring logits of one
// token, at any alignment (663 us for 128250 entries).
//
// Both CTAs' codes are counted by the leader's barriers, each CTA's scales by its
// own; its scale warps then arrive at the leader's `scaled`. The leader's commits
// go to both CTAs.
constexpr int kPairThreads = 768;
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = 2 * kWBytes + 3 * kSfTiles * kMxTileBytes;
constexpr int kPairSfCols = 3 * 4 * kSfTiles;  // M's 128 rows and N's 256
constexpr int kPairD = 256;
constexpr int kPairSmem = kPairStages * kPairStageBytes + 1024 + 512;
static_assert(kPairD + kPairStages * kPairSfCols <= 512, "tensor memory");
static_assert(kPairSmem <= kSmemBudget, "shared memory");

struct PairArgs {
  MxArgs c;
  const uint8_t* m_scales;  // of the operand whose rows are M, and N
  const uint8_t* n_scales;
  int m_row_tiles, n_row_tiles;  // 128-row tiles of either
  int units, token_units;        // tiles in all, and along the tokens
};

__device__ __forceinline__ void mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 bytes of logits. They go out of the L2 before the operands, which are read
// again: 636 us instead of 662 for 4096 tokens on 128256 x 4096.
__device__ __forceinline__ void store_sector(void* o, const uint32_t (&r)[8], uint64_t policy) {
  asm volatile("st.global.L1::no_allocate.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(o),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void store_sector(float* o, const float (&z)[8], uint64_t policy) {
  uint32_t r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(z[j]);
  store_sector(static_cast<void*>(o), r, policy);
}
__device__ __forceinline__ void store_sector(uint16_t* o, const float (&z)[16], uint64_t policy) {
  uint32_t r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = pack_bf16(z[2 * j], z[2 * j + 1]);
  store_sector(static_cast<void*>(o), r, policy);
}

// Arrives at a barrier of the pair's other CTA or its own. What this orders between
// the CTAs is tensor memory, for which tcgen05.fence::before_thread_sync stands in
// front; a release at cluster scope waits for the SM's memory traffic as well, 1300
// cycles a stage: 4096 tokens on 128256 x 4096 took 1430 us with it and 773 without.
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <bool TOKENS_M, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_m, const __grid_constant__ CUtensorMap map_n,
                        const __grid_constant__ PairArgs q) {
  constexpr int S = kPairStages;
  const MxArgs& p = q.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_m = smem;
  uint8_t* s_n = s_m + S * kWBytes;
  uint8_t* s_sf = s_n + S * kWBytes;  // per pair of stages: M's scale tiles, those of N's first 128 rows, of its other
  constexpr int kSfRun = 2 * kSfTiles * kMxTileBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_sf + S / 2 * 3 * kSfRun);
  uint64_t* sf_full = full + S / 2;
  uint64_t* scaled = sf_full + S / 2;  // the leader's: codes have landed and scales are in tensor memory, in both CTAs
  uint64_t* empty = scaled + S / 2;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 1;
  uint64_t* mma_done = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());

  // (the first wait can run out seconds after this, and all CTAs run at once)
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&empty[s], 1);
    for (int s = 0; s < S / 2; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&sf_full[s], 1);
      mbar_init(&scaled[s], 2 * 4);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * 16);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_m);
    tma_prefetch_desc(&map_n);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int k_pairs = (p.k_iters + 1) / 2;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);

  if (warp == 0 || warp == 22) {
    // Codes of M, of N: one warp for all copies of a stage took 670 cycles to issue them.
    const bool is_m = warp == 0;
    const CUtensorMap* map = is_m ? &map_m : &map_n;
    uint8_t* to = is_m ? s_m : s_n;
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0;
    bool aborted = false;
    for (int t = first; t < q.units && !aborted; t += step) {
      const int vu = t / q.token_units, tu = t - vu * q.token_units;  // a tile of W meets all tokens while in the L2
      const int row = ((is_m == TOKENS_M ? tu : vu) * 2 + rank) * 128;
      for (int k = 0; k < 2 * k_pairs; ++k) {
        if (!warp_wait(&empty[stage], phase ^ 1u, wc)) {
          aborted = true;
          break;
        }
        if (k < p.k_iters && elect_one()) {
          if (is_m && rank == 0 && (k & 1) == 0)
            mbar_arrive_expect_tx(&full[stage / 2], min(2, p.k_iters - k) * 4 * kWBytes);
          tma_load_2d_pair(to + stage * kWBytes, map, full0 + static_cast<uint32_t>(stage / 2) * 8u, k * kRowBytes, row);
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 23) {
    // Scales, for a pair of stages at once.
    int two = 0;
    uint32_t phase = 0;
    bool aborted = false;
    for (int t = first; t < q.units && !aborted; t += step) {
      const int vu = t / q.token_units, tu = t - vu * q.token_units;
      const int m_tile = 2 * (TOKENS_M ? tu : vu) + rank, n_tile = 2 * (TOKENS_M ? vu : tu);
      const int m_here = m_tile < q.m_row_tiles ? 1 : 0, n_here = min(2, q.n_row_tiles - n_tile);
      const uint8_t* m_from = q.m_scales + static_cast<int64_t>(m_tile) * p.k_tiles * kMxTileBytes;
      const uint8_t* n_from = q.n_scales + static_cast<int64_t>(n_tile) * p.k_tiles * kMxTileBytes;
      for (int k = 0; k < k_pairs; ++k) {
        if (!warp_wait(&empty[2 * two], phase ^ 1u, wc) || !warp_wait(&empty[2 * two + 1], phase ^ 1u, wc)) {
          aborted = true;
          break;
        }
        if (elect_one()) {
          uint8_t* s = s_sf + two * 3 * kSfRun;
          const uint32_t bytes = min(2 * kSfTiles, p.k_tiles - k * 2 * kSfTiles) * kMxTileBytes;
          mbar_arrive_expect_tx(&sf_full[two], bytes * (m_here + n_here));
          if (m_here) bulk_load(s, m_from + k * kSfRun, bytes, &sf_full[two]);
          bulk_load(s + kSfRun, n_from + k * kSfRun, bytes, &sf_full[two]);
          if (n_here > 1)
            bulk_load(s + 2 * kSfRun, n_from + p.k_tiles * kMxTileBytes + k * kSfRun, bytes, &sf_full[two]);
        }
        __syncwarp();
        if (++two == S / 2) {
          two = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int two = 0;  // the pair of stages
      uint32_t phase = 0, acc_phase = 0;
      const uint32_t m0 = smem_u32(s_m), n0 = smem_u32(s_n);
      bool aborted = false;
      for (int t = p.stall ? q.units : first; t < q.units && !aborted; t += step) {
        if (!warp_wait(tempty, acc_phase ^ 1u, wc)) break;
        acc_phase ^= 1u;
        tc_fence_after_sync();
        for (int k = 0; k < k_pairs; ++k) {
          if (!warp_wait(&scaled[two], phase, wc)) {
            aborted = true;
            break;
          }
          tc_fence_after_sync();
          if (elect_one()) {
            const int mmas = p.k_mmas - 2 * k * (kStageK / 64);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int stage = 2 * two + h;
              const uint32_t sf = tmem + static_cast<uint32_t>(kPairD + stage * kPairSfCols);
              const uint32_t a0 = m0 + stage * kWBytes, b0 = n0 + stage * kWBytes;
#pragma unroll
              for (int j = 0; j < kStageK / 64; ++j)
                if (h * (kStageK / 64) + j < mmas)
                  mma_mxf4_pair(tmem, sdesc_kmajor_sw128(a0 + j * 32), sdesc_kmajor_sw128(b0 + j * 32),
                                idesc_mxf4(256, 256, (j & 1) * 2), sf + 4 * (j >> 1), sf + 8 + 8 * (j >> 1),
                                (k | h | j) != 0 ? 1u : 0u);
              tc_commit_pair(&empty[stage], 0x3);
            }
            if (k == k_pairs - 1) tc_commit_pair(tfull, 0x3);
          }
          __syncwarp();
          if (++two == S / 2) {
            two = 0;
            phase ^= 1u;
          }
        }
      }
      if (elect_one()) {
        tc_commit_pair(mma_done, 0x1);
        wait_drain(mma_done, 0, p.timeout_ns, p.status);
      }
      __syncwarp();
    }
  } else if (warp < 6) {
    // Scales of a pair of stages whose copies have landed: its last MMAs are done,
    // since the loader waited for them, so its columns are free. The MMA warp has one
    // thing to wait for: each wait of its own showed in the time between its MMAs.
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t scaled0 = mapa_shared(smem_u32(scaled), 0);
    int two = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < q.units && ok; t += step) {
      for (int k = 0; k < k_pairs; ++k) {
        ok = warp_wait(&sf_full[two], phase, wc);
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (2 * k + h >= p.k_iters) break;
          const int stage = 2 * two + h;
          const uint32_t sf = t_lane + static_cast<uint32_t>(kPairD + stage * kPairSfCols);
          const uint8_t* m = s_sf + two * 3 * kSfRun + h * kSfTiles * kMxTileBytes + lane * 16;
          const uint8_t *n = m + kSfRun, *n2 = n + kSfRun;
          // (what was not loaded, of K or of rows, is an earlier use's bytes: not used, or not stored)
          store_scales2(sf, m, m + kMxTileBytes);
          // columns by K-tile, rows in order within one
          store_scales2(sf + 8, n, n2);
          store_scales2(sf + 16, n + kMxTileBytes, n2 + kMxTileBytes);
        }
        store_scales_wait();
        if (rank == 0) ok = warp_wait(&full[two], phase, wc);
        if (!ok) break;
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_pair(scaled0 + static_cast<uint32_t>(two) * 8u);
        if (++two == S / 2) {
          two = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    const int quarter = warp & 3, part = (warp - 6) >> 2;
    const uint32_t t_here = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * 64;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    const uint64_t policy = l2_policy_evict_first();
    uint32_t acc_phase = 0;
    for (int t = first; t < q.units; t += step) {
      const int vu = t / q.token_units, tu = t - vu * q.token_units;
      if (!warp_wait(tfull, acc_phase, wc)) break;
      acc_phase ^= 1u;
      tc_fence_after_sync();
      const int m = ((TOKENS_M ? tu : vu) * 2 + rank) * 128 + quarter * 32 + lane;
      uint32_t r[2][32];
      tmem_load_32cols(t_here, r[0]);
      tmem_load_32cols(t_here + 32, r[1]);
      tmem_load_wait_regs(r[0]);
      tmem_load_wait_regs(r[1]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_pair(tempty0);
      const int n = (TOKENS_M ? vu : tu) * 256 + part * 64;
      if (TOKENS_M && m < p.rows) {
        T* o = static_cast<T*>(p.out) + static_cast<int64_t>(m) * p.ld_out + n;
        constexpr int V = 32 / sizeof(T);
#pragma unroll
        for (int c = 0; c < 64; c += V) {
          float z[V];
#pragma unroll
          for (int j = 0; j < V; ++j) z[j] = finish(p, r[(c + j) / 32][(c + j) % 32]);
          if (n + c + V <= p.vocab) {
            store_sector(o + c, z, policy);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (n + c + j < p.vocab) o[c + j] = from_float<T>(z[j]);
          }
        }
      } else if (!TOKENS_M && m < p.vocab) {
        T* o = static_cast<T*>(p.out) + static_cast<int64_t>(n) * p.ld_out + m;
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (n + c < p.rows) o[c * p.ld_out] = from_float<T>(finish(p, r[c / 32][c % 32]));
      }
      __syncwarp();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) let_copies_land();
  __syncwarp();
  cluster_sync_all();  // neither CTA leaves while the other, or its copies, may still signal it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Codes as bytes [rows][cols / 2], boxes of 128 bytes x box_rows, 128-byte swizzle.
bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols / 2), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols / 2)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(kRowBytes), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Opts a kernel in to kSmemBudget on this device, once.
template <typename K>
int opt_in(K kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FLCE_ERR_CUDA;
  if (!(done.load() >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget) != cudaSuccess)
      return FLCE_ERR_CUDA;
    done.fetch_or(1ull << dev);
  }
  return FLCE_OK;
}

MxArgs arguments(const MxGemmParams& p) {
  MxArgs a = {};
  a.w_scales = p.w_scales;
  a.x_scales = p.a_scales;
  a.x = p.x;
  a.x_f32 = p.x_dtype == FLCE_DTYPE_F32;
  a.cols = static_cast<int>(p.cols);
  a.ld_x = p.ld_x;
  a.rows = static_cast<int>(p.rows);
  a.vocab = static_cast<int>(p.vocab);
  a.k_iters = static_cast<int>((p.cols + kStageK - 1) / kStageK);
  a.k_tiles = static_cast<int>((p.cols + kMxTileCols - 1) / kMxTileCols);
  a.k_mmas = static_cast<int>((p.cols + 63) / 64);
  a.v_tiles = static_cast<int>((p.vocab + kTileV - 1) / kTileV);
  a.out_mult = p.out_mult;
  a.softcap = p.softcap;
  a.inv_softcap = p.inv_softcap;
  a.out = p.out;
  a.ld_out = p.ld_out;
  a.status = p.status;
  a.timeout_ns = p.timeout_ns;
  a.stall = p.stall;
  return a;
}

template <int NT, bool RESIDENT, bool FUSED, typename T>
int run_tile(const MxGemmParams& p, int sms, cudaStream_t stream) {
  using P = Plan<NT, RESIDENT>;
  auto kernel = mx_gemm_kernel<NT, RESIDENT, FUSED, T>;
  static std::atomic<uint64_t> done{0};
  if (const int e = opt_in(kernel, done)) return e;
  CUtensorMap map_w, map_x;
  if (!encode_codes(&map_w, p.w_codes, p.vocab, p.cols, kTileV)) return FLCE_ERR_UNSUPPORTED;
  if (FUSED)
    map_x = map_w;  // not used
  else if (!encode_codes(&map_x, p.a_codes, p.rows, p.cols, NT))
    return FLCE_ERR_UNSUPPORTED;
  MxArgs a = arguments(p);
  a.stages = P::stages(a.k_iters);
  const int grid = a.v_tiles < sms ? a.v_tiles : sms;
  FLCE_LAUNCH(K_MX_GEMM, (kernel<<<grid, kThreads, P::smem(a.k_iters), stream>>>(map_w, map_x, a), cudaGetLastError()));
  return FLCE_OK;
}

template <bool TOKENS_M, typename T>
int run_pair(const MxGemmParams& p, int sms, cudaStream_t stream) {
  auto kernel = mx_gemm_pair_kernel<TOKENS_M, T>;
  static std::atomic<uint64_t> done{0};
  if (const int e = opt_in(kernel, done)) return e;
  CUtensorMap map_w, map_x;
  if (!encode_codes(&map_w, p.w_codes, p.vocab, p.cols, 128) || !encode_codes(&map_x, p.a_codes, p.rows, p.cols, 128))
    return FLCE_ERR_UNSUPPORTED;
  PairArgs q = {};
  q.c = arguments(p);
  const int x_tiles = static_cast<int>((p.rows + 127) / 128);
  q.m_scales = TOKENS_M ? p.a_scales : p.w_scales;
  q.n_scales = TOKENS_M ? p.w_scales : p.a_scales;
  q.m_row_tiles = TOKENS_M ? x_tiles : q.c.v_tiles;
  q.n_row_tiles = TOKENS_M ? q.c.v_tiles : x_tiles;
  q.token_units = (x_tiles + 1) / 2;
  const int64_t units = static_cast<int64_t>((q.c.v_tiles + 1) / 2) * q.token_units;
  if (units >= (1LL << 30)) return FLCE_ERR_ARG;
  q.units = static_cast<int>(units);
  const int clusters = q.units < sms / 2 ? q.units : sms / 2;
  FLCE_LAUNCH(K_MX_GEMM, (kernel<<<2 * clusters, kPairThreads, kPairSmem, stream>>>(
                              TOKENS_M ? map_x : map_w, TOKENS_M ? map_w : map_x, q), cudaGetLastError()));
  return FLCE_OK;
}

// One tile of tokens, with A resident if it fits beside a ring of four stages.
template <int NT>
bool resident(int64_t cols) {
  return Plan<NT, true>::stages(static_cast<int>((cols + kStageK - 1) / kStageK)) > 0;
}
template <int NT, typename T>
int run_few(const MxGemmParams& p, int sms, cudaStream_t s) {
  if constexpr (NT <= 64)
    if (p.x) return run_tile<NT, true, true, T>(p, sms, s);
  if (resident<NT>(p.cols)) return run_tile<NT, true, false, T>(p, sms, s);
  return run_tile<NT, false, false, T>(p, sms, s);
}

template <typename T>
int run_typed(const MxGemmParams& p, int sms, cudaStream_t s) {
  if (p.rows <= 16) return run_few<16, T>(p, sms, s);
  if (p.rows <= 32) return run_few<32, T>(p, sms, s);
  if (p.rows <= 64) return run_few<64, T>(p, sms, s);
  if (p.rows <= 128) return run_few<128, T>(p, sms, s);
  if (reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.ld_out * sizeof(T) % 32 == 0) return run_pair<true, T>(p, sms, s);
  return run_pair<false, T>(p, sms, s);
}

}  // namespace

bool mx_gemm_encodes(int64_t rows, int64_t cols) {
  if (rows > 64 || rows * cols > kMostFused) return false;
  return rows <= 16 ? resident<16>(cols) : rows <= 32 ? resident<32>(cols) : resident<64>(cols);
}

int launch_mx_gemm(const MxGemmParams& p, int sms, cudaStream_t s) {
  if (!load_encoder()) return FLCE_ERR_UNSUPPORTED;
  return p.out_dtype == FLCE_DTYPE_F32 ? run_typed<float>(p, sms, s) : run_typed<uint16_t>(p, sms, s);
}

}  // namespace flce
