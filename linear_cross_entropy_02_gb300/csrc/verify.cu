// Verification of drafted tokens against the target's distribution, from given random
// numbers: draft i is accepted while u_i q(d_i) < p(d_i), and one token more is drawn,
// from what p has above q at the first draft that is not accepted, from p itself if all
// were. That way the tokens are distributed as if the target had drawn them itself.
//
// Two kernels. The first finds what the filters keep of every row, and the kept weights'
// sum, with the kernels of sampling (sample_device.cuh), so that p and q are exactly the
// distributions that flce_sample draws from. The second takes a request: it compares the
// drafts, and goes over one row of the target and one of the draft to draw the last token.
// That row's weights are whole multiples of 2^-40, as in sampling: sums do not depend on
// the order or on how many CTAs share a row. Few requests are spread over clusters. The second kernel is launched
// while the first still ends, and waits for it: 2 of 98 us for a large batch. (It follows the first CTAs to end of
// the kernel for rows without filters, whose are small; beside sampling's, which fill an SM each, it would
// come to lie on few SMs: 47 us for 33 requests of mixed settings, 43 so.)
#include "model_internal.h"
#include "sample_device.cuh"

namespace flce {

namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

// What became of a request's drafts.
enum Stop { kAccepted = -1, kRejected, kNoDraft, kBad };

struct VerifyShared {
  uint64_t seg_weight[kSegments];
  uint64_t totals[kMaxCluster];  // of the CTAs' slices
  uint64_t goal;
  int count;
  int stop;
};

__device__ __forceinline__ uint64_t f2_fma_rz(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two logits at a time: packed arithmetic rounds each half as the single instruction does.
struct Pairs {
  uint64_t minus_top, inv;
  __device__ __forceinline__ Pairs(float top, float inverse) : minus_top(f2_pack(-top, -top)), inv(f2_pack(inverse, inverse)) {}
  __device__ __forceinline__ uint64_t exponentials(float x0, float x1) const {
    float t0, t1;
    f2_unpack(f2_mul(f2_add(f2_pack(x0, x1), minus_top), inv), t0, t1);
    return f2_pack(expf(t0), expf(t1));
  }
  // halves() of two exponentials, 2^23 above each half: a for the upper ones, b for the lower.
  __device__ __forceinline__ static void split(uint64_t e, uint64_t& a, uint64_t& b) {
    const uint64_t scale = f2_pack(1048576.f, 1048576.f), large = f2_pack(8388608.f, 8388608.f), minus = f2_pack(-1.f, -1.f);
    a = f2_fma_rz(e, scale, large);
    b = f2_fma_rz(f2_fma(e, scale, f2_fma(a, minus, large)), scale, large);
  }
  // the whole weights as numbers over the sum
  __device__ __forceinline__ static uint64_t shares(uint64_t e, uint64_t over) {
    uint64_t a, b;
    split(e, a, b);
    const uint64_t less = f2_pack(-8388608.f, -8388608.f);
    return f2_mul(f2_fma(f2_add(a, less), f2_pack(1048576.f, 1048576.f), f2_add(b, less)), over);
  }
};
constexpr uint32_t kLarge = 0x4B000000u;  // bits of 2^23

// A row's distribution: whole weights of its logits.
struct Kept {
  RowCut c;
  uint32_t last_key;  // the last kept logit's order key, complemented; ties are cut by index
  float least;        // no logit below it is kept
  bool all;           // all are
  __device__ __forceinline__ Kept(const RowCut& cut) : c(cut), last_key(static_cast<uint32_t>(cut.last >> 32)) {
    all = c.last == ~0ull && !(c.min_p > 0.f);
    least = c.last == ~0ull ? -INFINITY : key_value(~last_key);
  }
  // The exponential, 0 for what is not kept.
  __device__ __forceinline__ float exponential(float x, uint32_t index) const {
    const float e = expf(__fmul_rn(x - c.top, c.inv));
    if (all) return e;
    const uint32_t k = ~order_key(x);
    const bool keep = k < last_key || (k == last_key && index <= static_cast<uint32_t>(c.last));
    return keep && e >= c.min_p ? e : 0.f;
  }
  __device__ __forceinline__ Halves weight(float x, uint32_t index) const { return halves(exponential(x, index)); }
  // The whole weight, as a number (it has at most 24 bits), over the sum.
  __device__ __forceinline__ float share(float x, uint32_t index) const {
    const float e = exponential(x, index);
    const float a = __fmaf_rz(e, 1048576.f, 8388608.f);
    const float b = __fmaf_rz(__fmaf_rn(e, 1048576.f, 8388608.f - a), 1048576.f, 8388608.f);
    return __fmul_rn(fmaf(a - 8388608.f, 1048576.f, b - 8388608.f), c.over);
  }
  __device__ __forceinline__ double probability(float x, uint32_t index) const {
    const Halves w = weight(x, index);
    return __ddiv_rn(__ll2double_rn((static_cast<int64_t>(w.hi) << 20) + w.lo), __ll2double_rn(static_cast<int64_t>(c.whole)));
  }
  __device__ __forceinline__ float logprob(float x) const {
    return __fmul_rn(x - c.top, c.inv) - logf(__ll2float_rn(static_cast<int64_t>(c.whole)) * (1.f / kFixed));
  }
};

// What becomes of draft d, given the target's logit x and the draft's logit y for it (`g` is
// not used without a draft's row): kAccepted, kRejected or kBad.
__device__ __forceinline__ int compare(const RowCut& t, const RowCut& g, bool drawn, float x, float y, uint32_t d, float u) {
  if (t.whole == 0 || u != u || (drawn && g.whole == 0)) return kBad;
  // p and q in 32 bits are within 2^-22 of theirs: only where u q comes near p does it take
  // double precision, which this chip has little of (two divisions are some microseconds)
  const Kept target(t);
  const float p32 = target.share(x, d), uq = u * (drawn ? Kept(g).share(y, d) : 1.f);
  bool less = uq < p32;
  if (fabsf(uq - p32) <= 0x1p-20f * p32)
    less = __dmul_rn(static_cast<double>(u), drawn ? Kept(g).probability(y, d) : 1.0) < target.probability(x, d);
  return less ? kAccepted : kRejected;
}

// ---------------------------------------------------------------- rows without filters
// Their kept set is the row, so only its maximum and the sum of its weights are wanted:
// one pass, with the slice of the row in registers between the two. A cluster per row, of
// as many CTAs as its registers need, several of them on an SM so that one loads while the
// others add up. 64 requests of 5 drafts on 129280 bf16, 704 rows, take 74 us (2.5 TB/s), 66 where those behind
// a draft that is not accepted are left out (40% of them), some 115 with sampling's kernel: 19 instructions a
// logit, half of them the exponential, fill 62% of the issue slots.
constexpr int kPlainVecs = 8, kPlainWarps = 16;  // (of the larger CTAs)

__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b, const uint16_t*) {  // bf16 pairs
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b, const float*) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  return __float_as_uint(r);
}

// Rows behind a draft that is not accepted are not wanted. Where there are more rows than run at
// once they go by place, all requests' first rows first, and whoever completes a draft's rows compares
// it: rows that start later than that leave their work. (A hint: a CTA that comes too early to see it
// works in vain, and what such rows leave in p.cuts is not looked at.)
struct Progress {
  uint32_t* stopped;  // [batch] drafts + 1 - place of the first draft known not to be accepted, 0 if none is
  uint32_t* rows;     // [batch][drafts] rows that are summed
};

// What the writer of row (request, place)'s cut does then.
template <typename T>
__device__ void row_is_summed(const VerifyParams& p, const Progress& progress, int64_t request, int place) {
  if (place >= p.drafts) return;
  __threadfence();
  if (atomicAdd(&progress.rows[request * p.drafts + place], 1u) + 1 < (p.draft ? 2u : 1u)) return;
  __threadfence();
  const int64_t d = __ldg(p.draft_tokens + request * p.drafts + place);
  if (d < 0 || d >= p.vocab) return;
  auto cut = [](const RowCut* from) {  // past the L1
    union {
      uint4 u[2];
      RowCut c;
    } v;
    static_assert(sizeof(RowCut) == 32, "two vectors");
    v.u[0] = __ldcg(reinterpret_cast<const uint4*>(from));
    v.u[1] = __ldcg(reinterpret_cast<const uint4*>(from) + 1);
    return v.c;
  };
  const RowCut t = cut(p.cuts + request * (p.drafts + 1) + place);
  const RowCut g = p.draft ? cut(p.cuts + p.target_rows + request * p.drafts + place) : t;
  const float x = to_float<T>(static_cast<const T*>(p.x)[request * p.batch_ld + place * p.ld + d]);
  const float y = p.draft ? to_float<T>(static_cast<const T*>(p.draft)[request * p.draft_batch_ld + place * p.draft_ld + d]) : 0.f;
  if (compare(t, g, p.draft != nullptr, x, y, static_cast<uint32_t>(d), p.u[request * (p.drafts + 1) + place]) != kAccepted)
    atomicMax(&progress.stopped[request], static_cast<uint32_t>(p.drafts + 1 - place));
}

struct PlainShared {
  uint32_t tops[kMaxCluster];
  unsigned long long totals[kMaxCluster];
  uint32_t keys[kPlainWarps];
  unsigned long long sums[kPlainWarps];
};

template <typename T, int kPlainThreads>
__global__ void __launch_bounds__(kPlainThreads, 1024 / kPlainThreads) verify_plain_kernel(const VerifyParams p, const int slice, const Progress progress) {
  __shared__ PlainShared s;
  constexpr int E = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // all are running before the first write into another
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // they wait for this grid's end
  uint32_t r = blockIdx.x / ctas;  // (32 bits: divisions of 64 are a hundred instructions)
  if (progress.stopped) {
    // by place: a request's row of the target, then its row of the draft, then the next request's
    const uint32_t drafts = static_cast<uint32_t>(p.drafts), target_rows = static_cast<uint32_t>(p.target_rows);
    const uint32_t batch = target_rows / (drafts + 1), kinds = p.draft ? 2 : 1, at_place = r / (batch * kinds);
    const uint32_t at = r - at_place * batch * kinds;
    if (at_place >= drafts)  // of the target alone
      r = at * (drafts + 1) + at_place;
    else
      r = at % kinds ? target_rows + at / kinds * drafts + at_place : at / kinds * (drafts + 1) + at_place;
  }
  const T* start;
  int64_t request;
  int place;
  if (!verify_row(p, r, &start, &request, &place)) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    return;
  }
  // (the row's CTAs may see different answers here: all go through the barriers)
  bool wanted = true;
  if (progress.stopped) {
    const uint32_t stop = __shfl_sync(0xffffffffu, *static_cast<volatile uint32_t*>(progress.stopped + request), 0);
    wanted = stop == 0 || place <= static_cast<int>(p.drafts + 1 - stop);
  }
  const int vocab = static_cast<int>(p.vocab), c0 = static_cast<int>(rank) * slice, size = max(0, min(slice, vocab - c0));
  start += c0;
  const bool aligned = reinterpret_cast<uintptr_t>(start) % 16 == 0;
  Raw<T, E> raw[kPlainVecs];
  uint32_t key = 0;
  if (wanted) {
#pragma unroll
    for (int j = 0; j < kPlainVecs; ++j) {
      const int v = static_cast<int>(threadIdx.x) + j * kPlainThreads;
      if (aligned && (v + 1) * E <= size) {
        raw[j] = load_raw<T, E>(start + v * E);
      } else {
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = v * E + e < size ? to_float<T>(start[v * E + e]) : -INFINITY;
        raw[j] = pack<T, E>(x);
      }
    }
    // the largest logit, NaN if there is one
    uint32_t most = raw[0].u.x;
#pragma unroll
    for (int j = 0; j < kPlainVecs; ++j) {
      const uint32_t w[4] = {raw[j].u.x, raw[j].u.y, raw[j].u.z, raw[j].u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) most = max_nan(most, w[i], static_cast<const T*>(nullptr));
    }
    float mine = __uint_as_float(most);
    if constexpr (sizeof(T) == 2) mine = __uint_as_float(max_nan(most << 16, most & 0xFFFF0000u, static_cast<const float*>(nullptr)));
    // (a NaN, made positive, ranks above infinity)
    key = mine != mine ? 0xFFFFFFFFu : order_key(mine);
  }
  key = __reduce_max_sync(0xffffffffu, key);
  if (lane == 0) s.keys[warp] = key;
  __syncthreads();
  key = __reduce_max_sync(0xffffffffu, s.keys[lane % (kPlainThreads / 32)]);
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (threadIdx.x < ctas) remote_store(&s.tops[rank], threadIdx.x, key);
  row_barrier<true>();
  for (uint32_t c = 0; c < ctas; ++c) key = max(key, s.tops[c]);
  const float top = key_value(key);
  const bool bad = !(fabsf(top) < INFINITY);
  const float inv = fmaxf(1.f / p.temperature, kLeast);
  // Weights in halves, as halves() takes them; what it subtracts from each comes off the sums.
  Sum sum;
  if (wanted) {
    const Pairs pairs(top, inv);
#pragma unroll
    for (int j = 0; j < kPlainVecs; ++j) {
      float x[E];
      unpack<T, E>(raw[j], x);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        uint64_t a, b;
        Pairs::split(pairs.exponentials(x[e], x[e + 1]), a, b);
        sum.hi += static_cast<uint32_t>(a) + static_cast<uint32_t>(a >> 32);
        sum.lo += static_cast<uint32_t>(b) + static_cast<uint32_t>(b >> 32);
      }
    }
    constexpr uint32_t kLess = static_cast<uint32_t>(uint64_t{kLarge} * (kPlainVecs * E));
    sum.hi -= kLess;
    sum.lo -= kLess;
  }
  const uint64_t mine = sum.total();
  if (lane == 0) s.sums[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const uint64_t all = warp_total(lane < kPlainThreads / 32 ? s.sums[lane] : 0);
    if (lane == 0)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s.totals[rank]), 0)), "l"(all) : "memory");
  }
  row_barrier<true>();
  if (rank == 0 && threadIdx.x == 0) {
    uint64_t whole = 0;
    for (uint32_t c = 0; c < ctas; ++c) whole += s.totals[c];
    p.cuts[r] = {~0ull, bad ? 0 : whole, top, inv, 0.f, bad ? 0.f : reciprocal(whole)};
    if (progress.stopped) row_is_summed<T>(p, progress, request, place);
  }
}

// Logits that a CTA's registers hold.
template <typename T>
constexpr int64_t plain_slice(int threads) {
  return int64_t{threads} * kPlainVecs * (16 / static_cast<int64_t>(sizeof(T)));
}

// Whether no row has a filter, as far as the host knows, and a cluster's registers hold one.
template <typename T>
bool plain_rows(const VerifyParams& p) {
  if (p.temperatures || p.top_ks || p.top_ps || p.min_ps) return false;
  if (!(p.temperature > 0.f) || 1.f / p.temperature > 3e38f || p.top_p < 1.f || p.min_p > 0.f) return false;
  return (p.top_k <= 0 || p.top_k >= p.vocab) && p.vocab <= kMaxCluster * plain_slice<T>(512);
}

template <typename T, int kPlainThreads>
cudaError_t run_plain(const VerifyParams& p, int sms, cudaStream_t s) {
  // few rows are spread further, down to 4096 logits per CTA
  int ctas = 1;
  while (ctas * plain_slice<T>(kPlainThreads) < p.vocab ||
         (ctas < kMaxCluster && p.rows * ctas * 2 <= 1024LL / kPlainThreads * sms && p.vocab / ctas > 4096))
    ctas *= 2;
  const int slice = static_cast<int>(((p.vocab + ctas - 1) / ctas + 63) / 64 * 64);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * ctas));
  cfg.blockDim = dim3(kPlainThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  Progress progress = {};
  if (p.rows * ctas > 1024LL / kPlainThreads * sms && p.drafts > 0) {
    const int64_t batch = p.target_rows / (p.drafts + 1);
    progress = {p.progress, p.progress + batch};
    const cudaError_t e = cudaMemsetAsync(p.progress, 0, sizeof(uint32_t) * batch * (p.drafts + 1), s);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, verify_plain_kernel<T, kPlainThreads>, p, slice, progress);
}

// Smaller CTAs, four on an SM, where eight of them hold a row: 704 rows of 129280 bf16 74 us, 78 with the larger ones.
template <typename T>
cudaError_t run_plain_typed(const VerifyParams& p, int sms, cudaStream_t s) {
  return p.vocab <= kMaxCluster * plain_slice<T>(256) ? run_plain<T, 256>(p, sms, s) : run_plain<T, 512>(p, sms, s);
}

// ---------------------------------------------------------------- a request
template <typename T, bool MULTI>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyParams p, int64_t* accepted, const int slice) {
  __shared__ VerifyShared s;
  constexpr int E = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank = 0, ctas = 1;
  if constexpr (MULTI) {
    rank = cluster_ctarank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // all are running before the first write into another
  }
  // this grid is launched while the one before it, which writes p.cuts, may still run
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t b = blockIdx.x / ctas, K = p.drafts;
  const T* target = static_cast<const T*>(p.x) + b * p.batch_ld;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + b * p.draft_batch_ld : nullptr;
  const int64_t* drafts = p.draft_tokens + b * K;
  const float* u = p.u + b * (K + 1);
  const RowCut* cuts = p.cuts + b * (K + 1);
  const RowCut* draft_cuts = p.cuts + p.target_rows + b * K;
  int64_t* tokens = p.tokens + b * (K + 1);
  float* logprobs = p.logprobs ? p.logprobs + b * (K + 1) : nullptr;

  // ---- the drafts, a lane each
  if (warp == 0) {
    int count = 0, stop = kNoDraft;
    for (int64_t base = 0; base < K; base += 32) {
      const int64_t i = base + lane;
      int mine = kAccepted;
      const uint32_t none = __ballot_sync(0xffffffffu, i < K && !(drafts[i] >= 0 && drafts[i] < p.vocab));
      if (i < K) {
        const int64_t d = drafts[i];
        // (an earlier lane without a draft: this row was not looked at)
        if (none & ((2u << lane) - 1u)) {
          mine = kNoDraft;
        } else {
          const RowCut t = cuts[i], g = draft ? draft_cuts[i] : t;
          const float x = to_float<T>(target[i * p.ld + d]), y = draft ? to_float<T>(draft[i * p.draft_ld + d]) : 0.f;
          mine = compare(t, g, draft != nullptr, x, y, static_cast<uint32_t>(d), u[i]);
          if (mine == kAccepted && rank == 0 && logprobs) logprobs[i] = Kept(t).logprob(x);
        }
      }
      const uint32_t stopped = __ballot_sync(0xffffffffu, mine >= 0);
      if (stopped) {
        const int first = __ffs(stopped) - 1;
        stop = __shfl_sync(0xffffffffu, mine, first);
        count += first;
        break;
      }
      count += static_cast<int>(K - base < 32 ? K - base : 32);
    }
    if (lane == 0) {
      s.count = count;
      s.stop = stop;
    }
  }
  __syncthreads();
  const int n = s.count;
  int stop = s.stop;
  const float v = u[K];
  if (stop != kBad && (cuts[n].whole == 0 || v != v)) stop = kBad;
  if (rank == 0) {
    for (int64_t i = threadIdx.x; i <= K; i += kVerifyThreads) {
      if (i == n && stop != kBad) continue;  // the drawn token's place
      tokens[i] = i < n ? drafts[i] : -1;
      if (logprobs && i >= n) logprobs[i] = i > n ? 0.f : __uint_as_float(0x7FC00000u);
    }
    if (threadIdx.x == 0) accepted[b] = n;
  }
  if (stop == kBad) {
    if constexpr (MULTI) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    return;
  }

  // ---- the token behind them
  const Kept kept(cuts[n]);
  const T* row = target + n * p.ld;
  const T* other = stop == kRejected && draft ? draft + n * p.draft_ld : nullptr;
  const Kept drafted(other ? draft_cuts[n] : cuts[n]);
  const uint32_t rejected = stop == kRejected ? static_cast<uint32_t>(drafts[n]) : 0u;
  const int vocab = static_cast<int>(p.vocab), c0 = static_cast<int>(rank) * slice, size = max(0, min(slice, vocab - c0));
  const int vecs = (size + E - 1) / E;
  const bool aligned = reinterpret_cast<uintptr_t>(row) % 16 == 0 && (!other || reinterpret_cast<uintptr_t>(other) % 16 == 0);
  bool rest = stop == kRejected;  // draw from max(p - q, 0)
  const bool whole_rows = kept.all && drafted.all;  // nothing is cut
  const uint64_t share = f2_pack(kept.c.over, kept.c.over), other_share = f2_pack(drafted.c.over, drafted.c.over);
  const Pairs kept_pairs(kept.c.top, kept.c.inv), other_pairs(drafted.c.top, drafted.c.inv);
  auto read = [&](const T* from, int vec, float (&x)[E]) {
    if (aligned && (vec + 1) * E <= size) {
      unpack<T, E>(load_raw<T, E>(from + c0 + vec * E), x);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = vec * E + e < size ? to_float<T>(from[c0 + vec * E + e]) : -INFINITY;
    }
  };
  // (most of a filtered row's vectors hold nothing that is kept)
  auto weights = [&](int vec, Halves (&w)[E]) {
    float x[E], y[E];
    read(row, vec, x);
    float most = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) most = fmaxf(most, x[e]);
    if (most < kept.least) {
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = {0u, 0u};
      return;
    }
    const uint32_t first = static_cast<uint32_t>(c0 + vec * E);
    if (whole_rows) {
      if (other) read(other, vec, y);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        uint64_t v = kept_pairs.exponentials(x[e], x[e + 1]), a, b;
        if (rest) {
          v = Pairs::shares(v, share);
          const uint64_t q = other ? Pairs::shares(other_pairs.exponentials(y[e], y[e + 1]), other_share)
                                   : f2_pack(first + e == rejected ? 1.f : 0.f, first + e + 1 == rejected ? 1.f : 0.f);
          float r0, r1;
          f2_unpack(f2_fma(q, f2_pack(-1.f, -1.f), v), r0, r1);  // (one rounding: of the difference)
          v = f2_pack(__saturatef(r0), __saturatef(r1));
        }
        Pairs::split(v, a, b);
        w[e] = {static_cast<uint32_t>(a) - kLarge, static_cast<uint32_t>(b) - kLarge};
        w[e + 1] = {static_cast<uint32_t>(a >> 32) - kLarge, static_cast<uint32_t>(b >> 32) - kLarge};
      }
      return;
    }
    if (!rest) {
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = kept.weight(x[e], first + e);
      return;
    }
    if (other) read(other, vec, y);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float q = other ? drafted.share(y[e], first + e) : first + e == rejected ? 1.f : 0.f;
      w[e] = halves(__saturatef(__fsub_rn(kept.share(x[e], first + e), q)));
    }
  };
  const int per = Row<T, kVerifyThreads>::segment_vecs(vecs), segs = (vecs + per - 1) / per;
  if constexpr (MULTI) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  uint64_t total, before;
  while (true) {
    for (int i = threadIdx.x; i < kSegments; i += kVerifyThreads)
      if (i >= segs) s.seg_weight[i] = 0;
    for (int seg = warp; seg < segs; seg += kVerifyWarps) {
      Sum acc;
      const int v1 = min((seg + 1) * per, vecs);
      for (int vec = seg * per + lane; vec < v1; vec += 32) {
        Halves w[E];
        weights(vec, w);
#pragma unroll
        for (int e = 0; e < E; ++e) acc.add(w[e]);
      }
      const uint64_t sum = acc.total();
      if (lane == 0) s.seg_weight[seg] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      uint64_t sum = 0;
      for (int i = lane; i < kSegments; i += 32) sum += s.seg_weight[i];
      sum = warp_total(sum);
      if (lane < static_cast<int>(ctas)) {
        if constexpr (MULTI)
          asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s.totals[rank]), lane)), "l"(sum) : "memory");
        else
          s.totals[0] = sum;
      }
    }
    row_barrier<MULTI>();
    total = before = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
      if (c < rank) before += s.totals[c];
      total += s.totals[c];
    }
    if (total > 0 || !rest) break;
    // p nowhere above q, as far as whole multiples of 2^-40 show it: from p itself
    rest = false;
    row_barrier<MULTI>();  // the totals have been read by all
  }
  // ---- the first token whose running sum is above u times the whole
  if (warp != 0) return;
  if (lane == 0) s.goal = answer_goal(v, total);
  __syncwarp();
  const uint64_t goal = s.goal;
  if (goal < before || goal >= before + s.totals[rank]) return;
  int found = 0;
  for (int base = 0; base < kSegments; base += 32) {
    const uint64_t w = s.seg_weight[base + lane], inc = warp_inclusive(w);
    const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > goal);
    if (hit) {
      const int at = __ffs(hit) - 1;
      found = base + at;
      before += __shfl_sync(0xffffffffu, inc - w, at);
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  const int v1 = min((found + 1) * per, vecs);
  for (int base = found * per; base < v1; base += 32) {
    const int vec = base + lane;
    Halves w[E];
    uint64_t sum = 0;
    if (vec < v1) {
      weights(vec, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += (static_cast<uint64_t>(w[e].hi) << 20) + w[e].lo;
    }
    const uint64_t inc = warp_inclusive(sum);
    uint64_t run = before + inc - sum;
    if (run <= goal && goal < run + sum) {
      float x[E];
      read(row, vec, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint64_t we = (static_cast<uint64_t>(w[e].hi) << 20) + w[e].lo;
        if (run <= goal && goal < run + we) {
          tokens[n] = c0 + vec * E + e;
          if (logprobs) logprobs[n] = kept.logprob(x[e]);
        }
        run += we;
      }
    }
    if (__any_sync(0xffffffffu, goal < before + __shfl_sync(0xffffffffu, inc, 31))) break;
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
}

template <typename T, bool MULTI>
cudaError_t run_verify(const VerifyParams& p, int64_t batch, int64_t* accepted, int ctas, cudaStream_t s) {
  const int slice = static_cast<int>(((p.vocab + ctas - 1) / ctas + 63) / 64 * 64);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch * ctas));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, MULTI>, p, accepted, slice);
}

template <typename T>
cudaError_t run_verify_typed(const VerifyParams& p, int64_t batch, int64_t* accepted, int sms, cudaStream_t s) {
  int ctas = 1;
  while (ctas < kMaxCluster && batch * ctas * 2 <= 2LL * sms && p.vocab / ctas > 4096) ctas *= 2;
  return ctas > 1 ? run_verify<T, true>(p, batch, accepted, ctas, s) : run_verify<T, false>(p, batch, accepted, 1, s);
}

}  // namespace

cudaError_t launch_verify_cuts(const VerifyParams& p, int sms, cudaStream_t s) {
  if (p.dtype == FLCE_DTYPE_F32) return plain_rows<float>(p) ? run_plain_typed<float>(p, sms, s) : run_typed<float, true>(p, sms, s);
  return plain_rows<uint16_t>(p) ? run_plain_typed<uint16_t>(p, sms, s) : run_typed<uint16_t, true>(p, sms, s);
}

cudaError_t launch_verify(const VerifyParams& p, int64_t batch, int64_t* accepted, int sms, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? run_verify_typed<float>(p, batch, accepted, sms, s) : run_verify_typed<uint16_t>(p, batch, accepted, sms, s);
}

}  // namespace flce
