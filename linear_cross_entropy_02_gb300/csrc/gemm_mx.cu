// out = cap(m A W^T) of microscaled 4-bit operands on the tensor cores:
// tcgen05.mma kind::mxf4 with a power-of-two scale per 32 elements, products
// summed in fp32 in tensor memory.
//
// W's rows are the M dimension (128 vocabulary entries per tile) and the tokens
// the N dimension, so that one token and a whole prompt run through the same
// kernel: for a few tokens the tile is 128 x 16 and the kernel streams W once
// through a deep ring of TMA copies, bound by HBM; for a prompt it is 128 x 192
// and bound by the tensor cores and the L2. A lane of tensor memory is then a
// vocabulary entry, and a warp's store for one token is one contiguous run of
// logits whatever the row stride's alignment.
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
// Warp 0 loads, warp 1 issues the MMAs, warps 2-5 store, warps 6-9 carry scales:
// two accumulators, so that the stores of one tile run under the MMAs of the
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
constexpr int64_t kMostFused = 40960;  // 4 tokens of 7168: 83.0 us so, 83.8 with a launch before; 8: 86.9 and 85

// Shared and tensor memory of a tile of NT tokens. RESIDENT: A's codes and scales
// stay in shared memory in front of the ring, which then holds W alone.
template <int NT, bool RESIDENT>
struct Plan {
  static constexpr int row_tiles = (NT + 127) / 128;  // 128-row scale tiles that the tokens can touch
  static constexpr int x_bytes = NT * kRowBytes;
  static constexpr int w_sf = kSfTiles * kMxTileBytes;
  static constexpr int x_sf = row_tiles * kSfTiles * kMxTileBytes;
  static constexpr int x_all = x_bytes + x_sf;  // of one stage's K
  static constexpr int stage = kWBytes + w_sf + (RESIDENT ? 0 : x_all);
  static constexpr int d_cols = NT < 32 ? 32 : NT;      // one accumulator
  static constexpr int sf_cols = 4 * kSfTiles * (1 + row_tiles);
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
  int x_row_tiles;
  const void* x;  // FUSED: the tokens as they are
  int x_f32, cols;
  int64_t ld_x;
  int v_tiles, n_tiles, stages;
  float out_mult, softcap, inv_softcap;
  void* out;
  int64_t ld_out;
  int32_t* status;
  uint64_t timeout_ns;
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
// wait_bounded by a whole warp, which then agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, w));
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
  const int total = p.v_tiles * p.n_tiles;

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
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool aborted = false;
    if (RESIDENT && !FUSED && elect_one()) {  // one tile of tokens, whose scales are one row of tiles
      mbar_arrive_expect_tx(x_full, p.k_iters * P::x_bytes + p.k_tiles * kMxTileBytes);
      for (int k = 0; k < p.k_iters; ++k) tma_load_2d(s_x + k * P::x_bytes, &map_x, x_full, k * kRowBytes, 0);
      bulk_load(s_xsf, p.x_scales, static_cast<uint32_t>(p.k_tiles) * kMxTileBytes, x_full);
    }
    __syncwarp();
    for (int t = blockIdx.x; t < total && !aborted; t += gridDim.x) {
      const int vb = t / p.n_tiles, nb = t - vb * p.n_tiles;  // a tile of W meets all tokens while it is in the L2
      const int xt0 = nb * NT / 128;
      const int xts = min(P::row_tiles, p.x_row_tiles - xt0);
      for (int k = 0; k < p.k_iters; ++k) {
        if (!warp_wait(&empty[stage], phase ^ 1u, wc)) {
          aborted = true;
          break;
        }
        if (elect_one()) {
          const int kt = k * kSfTiles;
          const uint32_t sf = static_cast<uint32_t>(min(kSfTiles, p.k_tiles - kt)) * kMxTileBytes;
          mbar_arrive_expect_tx(&full[stage], kWBytes + sf + (RESIDENT ? 0 : P::x_bytes + sf * xts));
          tma_load_2d(s_w + stage * kWBytes, &map_w, &full[stage], k * kRowBytes, vb * kTileV);
          bulk_load(s_wsf + stage * P::w_sf, p.w_scales + (static_cast<int64_t>(vb) * p.k_tiles + kt) * kMxTileBytes,
                    sf, &full[stage]);
          if (!RESIDENT) {
            tma_load_2d(s_x + stage * P::x_bytes, &map_x, &full[stage], k * kRowBytes, nb * NT);
            for (int i = 0; i < xts; ++i)
              bulk_load(s_xsf + stage * P::x_sf + i * kSfTiles * kMxTileBytes,
                        p.x_scales + (static_cast<int64_t>(xt0 + i) * p.k_tiles + kt) * kMxTileBytes, sf, &full[stage]);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (aborted && lane == 0) {
      // loads that may still be in flight land before the shared memory goes away
      if (RESIDENT && !FUSED) wait_drain(x_full, 0, p.timeout_ns, p.status);
      const int n = issued < S ? issued : S;
      int s = stage;
      uint32_t ph = phase;
      for (int i = 0; i < n; ++i) {
        if (s == 0) {
          s = S - 1;
          ph ^= 1u;
        } else {
          --s;
        }
        wait_drain(&full[s], ph, p.timeout_ns, p.status);
      }
    }
  } else if (warp == 1) {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    const uint32_t w0 = smem_u32(s_w), x0 = smem_u32(s_x);
    bool aborted = RESIDENT && !warp_wait(x_full, 0, wc);
    for (int t = blockIdx.x; t < total && !aborted; t += gridDim.x) {
      const int nb = t % p.n_tiles;
      const uint32_t x_shift = static_cast<uint32_t>(nb * NT % 128 / 32);  // first 32-row group of the tokens
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
          const uint32_t sfx = sf + 4 * kSfTiles + x_shift;
          const uint32_t a0 = w0 + stage * kWBytes, b0 = x0 + (RESIDENT ? k : stage) * P::x_bytes;
          const int mmas = p.k_mmas - k * (kStageK / 64);
#pragma unroll
          for (int j = 0; j < kStageK / 64; ++j)
            if (j < mmas)
              mma_mxf4(d, sdesc_kmajor_sw128(a0 + j * 32), sdesc_kmajor_sw128(b0 + j * 32),
                       idesc_mxf4(kTileV, NT, (j & 1) * 2), sf + 4 * (j >> 1), sfx + 4 * (j >> 1) * P::row_tiles,
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
    for (int t = blockIdx.x; t < total && __all_sync(0xffffffffu, ok); t += gridDim.x) {
      for (int k = 0; k < p.k_iters; ++k) {
        ok = wait_bounded(&full[stage], phase, wc);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after_sync();
        const uint32_t sf = t_lane + static_cast<uint32_t>(2 * P::d_cols + stage * P::sf_cols);
        const uint8_t* w = s_wsf + stage * P::w_sf + lane * 16;
        // (a last stage of one tile carries the stage before's bytes in the other's place: not used)
        store_scales2(sf, w, w + kMxTileBytes);
        const uint8_t* x = s_xsf + (RESIDENT ? k : stage) * P::x_sf + lane * 16;
        if (P::row_tiles == 1) {
          store_scales2(sf + 8, x, x + kMxTileBytes);
        } else {
          // columns by K-tile, rows in order within one
          store_scales2(sf + 8, x, x + 2 * kMxTileBytes);
          store_scales2(sf + 16, x + kMxTileBytes, x + 3 * kMxTileBytes);
        }
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
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const int vb = t / p.n_tiles, nb = t - vb * p.n_tiles;
      const bool ok = wait_bounded(&tfull[acc], acc_phase, wc);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after_sync();
      const int v = vb * kTileV + quarter * 32 + lane;
      const int n0 = nb * NT;
      const int n_here = min(NT, p.rows - n0);
      for (int c = 0; c < n_here; c += 32) {
        uint32_t r[32];
        tmem_load_32cols(t_lane + acc * P::d_cols + c, r);
        tmem_load_wait_regs(r);
        T* o = static_cast<T*>(p.out) + static_cast<int64_t>(n0 + c) * p.ld_out + v;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (c + j < n_here && v < p.vocab) {
            float z = __uint_as_float(r[j]) * p.out_mult;
            if (p.softcap > 0.f) z = p.softcap * tanhf(z * p.inv_softcap);
            o[j * p.ld_out] = from_float<T>(z);
          }
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

template <int NT, bool RESIDENT, bool FUSED, typename T>
int run_tile(const MxGemmParams& p, int sms, cudaStream_t stream) {
  using P = Plan<NT, RESIDENT>;
  auto kernel = mx_gemm_kernel<NT, RESIDENT, FUSED, T>;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FLCE_ERR_CUDA;
  if (!(done.load() >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget) != cudaSuccess)
      return FLCE_ERR_CUDA;
    done.fetch_or(1ull << dev);
  }
  CUtensorMap map_w, map_x;
  if (!encode_codes(&map_w, p.w_codes, p.vocab, p.cols, kTileV)) return FLCE_ERR_UNSUPPORTED;
  if (FUSED)
    map_x = map_w;  // not used
  else if (!encode_codes(&map_x, p.a_codes, p.rows, p.cols, NT))
    return FLCE_ERR_UNSUPPORTED;
  MxArgs a;
  a.w_scales = p.w_scales;
  a.x_scales = p.a_scales;
  a.x = p.x;
  a.x_f32 = p.x_dtype == FLCE_DTYPE_F32;
  a.cols = static_cast<int>(p.cols);
  a.ld_x = p.ld_x;
  a.rows = static_cast<int>(p.rows);
  a.vocab = static_cast<int>(p.vocab);
  a.k_iters = static_cast<int>((p.cols + kStageK - 1) / kStageK);
  a.stages = P::stages(a.k_iters);
  a.k_tiles = static_cast<int>((p.cols + kMxTileCols - 1) / kMxTileCols);
  a.k_mmas = static_cast<int>((p.cols + 63) / 64);
  a.x_row_tiles = static_cast<int>((p.rows + 127) / 128);
  a.v_tiles = static_cast<int>((p.vocab + kTileV - 1) / kTileV);
  a.n_tiles = static_cast<int>((p.rows + NT - 1) / NT);
  a.out_mult = p.out_mult;
  a.softcap = p.softcap;
  a.inv_softcap = p.inv_softcap;
  a.out = p.out;
  a.ld_out = p.ld_out;
  a.status = p.status;
  a.timeout_ns = p.timeout_ns;
  // An MMA's scales start on an even column of tensor memory: token tiles other
  // than the first need 64 rows or a multiple of it.
  static_assert(NT % 64 == 0 || NT < 64, "even scale columns");
  if (a.n_tiles > 1 && NT % 64 != 0) return FLCE_ERR_ARG;
  const int64_t total = static_cast<int64_t>(a.v_tiles) * a.n_tiles;
  if (total >= (1LL << 31)) return FLCE_ERR_ARG;
  const int grid = static_cast<int>(total < sms ? total : sms);
  FLCE_LAUNCH(K_MX_GEMM, (kernel<<<grid, kThreads, P::smem(a.k_iters), stream>>>(map_w, map_x, a), cudaGetLastError()));
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
  return run_tile<192, false, false, T>(p, sms, s);
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
