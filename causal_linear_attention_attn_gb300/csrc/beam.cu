// Beam search over states: selection of the best continuations, and pools of states that follow them.
//
// Selection.  Of a group's W beams with scores s_w and logits l_{w,v} over V tokens, the k best by
//   s_w + l_{w,v} - log sum_v' e^{l_{w,v'}},
// ties to the lowest w V + v.  The sum is formed in 32 bits, as the other rows' sums are (its logarithm is off by 4e-7
// at most where measured; 64-bit exponentials, by count, would take this GPU milliseconds for 512 rows of 131072), and what is added
// and compared after it in 64 bits: scores of hundreds have no bits for that in 32.  Within a beam the
// order is that of the logits, so the k best of each row are enough; HBM bounds it: the logits once.
//
// A block takes a run of one row in chunks of 4096 values, its warps an eighth of each, without waiting for one
// another: a warp keeps 512 values in registers while the next ones are on their way, adds up their exponentials
// against its running maximum, and keeps a list of candidates for its k best.  The bound that lets values into the
// lists is the block's k-th best of the first chunk, or a warp's so far if that is better; before there is one, the k-th
// largest of the lanes' largest values, sorted across the lanes, is a value that at least k reach.  Lists are ranked by counting (every candidate against every other), not
// extracted one after another.  A second kernel, a block a group, joins the runs of a row and the rows of the group the
// same way in 64 bits.  512 rows of 131072 in bf16 in 66 us, 2.0 TB/s: issue slots bound it (67 % taken, 300 instructions
// per 512 values).  With barriers a chunk and a bound a warp it took 307 us, with 32 values a lane (fewer warps) 88.
//
// Reordering.  A beam's first child keeps the slot of its state in every pool; its other children get the
// slots of the group's childless beams, with a copy.  So the states move no more than they must, in place:
// what is read (kept slots) and what is written (freed ones) never meet.  192 rows of 573 KB in 39 us, 5.6 TB/s.
#include <algorithm>

#include "internal.h"
#include "selective.cuh"

namespace la {

__device__ unsigned int g_beam_status;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 16;                  // values a thread and chunk
constexpr int kChunk = kBeamChunk;        // values a chunk
static_assert(kChunk == kThreads * kPer, "a chunk is a block's values");
constexpr int kCap = 256;                 // candidates of a warp
constexpr int kMaxK = 64;

// NaN counts as -inf, inf as the largest finite number: infinite logits share the probability.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f); }
// e^(x - top), top finite
__device__ __forceinline__ float exp_under(float x, float top) { return exp2_approx((x - top) * kLog2e); }
// Clean floats in order as unsigned numbers, all above 0 (no value); -0 as 0: they are equal.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kMinusInf = 0x007fffffu;  // ordered(-inf)

struct Cand {
  uint32_t key, token;  // key 0: none
};
__device__ __forceinline__ bool before(const Cand &a, const Cand &b) {
  return a.key > b.key || (a.key == b.key && a.token < b.token);
}

// Values of the warp's lanes, largest first (bitonic).
__device__ __forceinline__ float warp_sort(float x, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      const bool down = (lane & size) == 0 || size == 32, low = (lane & o) == 0;
      x = (down == low) ? fmaxf(x, y) : fminf(x, y);
    }
  return x;
}

template <typename T>
struct Chunk {  // a thread's kPer values: groups of kVec neighbours (16 bytes), kThreads groups apart
  static constexpr int kVec = 16 / (int)sizeof(T), kVecs = kPer / kVec;
  uint4 a[kVecs];
  // from place `at` of a row of n values.  Rows off 16-byte borders are loaded value by value, to the same lanes: equal
  // rows have equal sums then, to the last bit, and their ties are ties.
  __device__ __forceinline__ void load(const T *row, long at, long n) {
    const T *p = row + at + threadIdx.x * kVec;
    if ((reinterpret_cast<uintptr_t>(row) & 15) == 0 && at + kChunk <= n) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) a[j] = __ldcs(reinterpret_cast<const uint4 *>(p + j * kThreads * kVec));
    } else {
      const int left = (int)min(n - at, (long)kChunk) - (int)threadIdx.x * kVec;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        a[j] = make_uint4(0u, 0u, 0u, 0u);
        T *e = reinterpret_cast<T *>(&a[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (j * kThreads * kVec + i < left) e[i] = p[j * kThreads * kVec + i];
      }
    }
  }
  __device__ __forceinline__ float value(int i) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a);
    if (sizeof(T) == 4) return __uint_as_float(w[i % (kVecs * 4)]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  // the place of value i behind the chunk's start
  __device__ __forceinline__ static int place(int i) { return ((i / kVec) * kThreads + (int)threadIdx.x) * kVec + i % kVec; }
};

struct RowSmem {
  Cand list[kWarps][kCap], best[kWarps][kMaxK];
  float top[kWarps], sum[kWarps];
  int count[kWarps], total;
  uint32_t bound;  // what at least k of the block's values reach, in order; 0: nothing yet
};

// The k best of a list of n, in order (key 0 behind the last); all of `threads` threads, of which this is number `at`.
__device__ __forceinline__ void rank_list(const Cand *list, int n, int k, Cand *best, int at, int threads) {
  for (int i = max(n, 0) + at; i < k; i += threads) best[i] = Cand{0u, 0u};
  for (int i = at; i < n; i += threads) {
    const Cand c = list[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += before(list[j], c);
    if (r < k) best[r] = c;
  }
}

// Places of the block's candidates, the k best of each warp, among all of them: put(candidate, its place).
template <typename Put>
__device__ __forceinline__ void place_candidates(const RowSmem &m, int k, Put &&put) {
  for (int i = threadIdx.x; i < kWarps * k; i += kThreads) {
    const Cand c = m.best[i / k][i % k];
    if (c.key == 0) continue;
    int r = 0;  // its places in the warps' lists together
    for (int w = 0; w < kWarps; ++w) {
      int lower = 0, upper = k;  // the first of the list that it is not behind
      while (lower < upper) {
        const int mid = (lower + upper) / 2;
        if (before(m.best[w][mid], c))
          lower = mid + 1;
        else
          upper = mid;
      }
      r += lower;
    }
    if (r < k) put(c, r);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const __grid_constant__ BeamProblem p, const __grid_constant__ BeamSplit s) {
  __shared__ RowSmem m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long row = blockIdx.x / s.runs;
  const int run = (int)(blockIdx.x - row * s.runs), k = p.k;
  Cand *out = reinterpret_cast<Cand *>(s.cands) + (row * s.runs + run) * k;
  float *stat = s.stats + (row * s.runs + run) * 2;
  const float score = p.scores[row];
  const bool dead = !(score > -INFINITY), done = p.finished && p.finished[row];
  if (dead || done) {  // one continuation at no cost, or none: the rest are -inf, lowest token first
    if (tid == 0) stat[0] = run == 0 && !dead ? 0.f : -INFINITY, stat[1] = run == 0 && !dead ? 1.f : 0.f;
    if (tid < k) {
      Cand c{0u, 0u};
      if (run == 0) {
        const int first = dead ? 0 : 1;
        if (tid < first) {
          c = Cand{ordered(0.f), (uint32_t)p.eos};
        } else {
          uint32_t t = (uint32_t)(tid - first);
          if (!dead && t >= (uint32_t)p.eos) ++t;
          if (t < (uint32_t)p.V) c = Cand{kMinusInf, t};
        }
      }
      out[tid] = c;
    }
    return;
  }
  const T *logits = (const T *)p.logits + row * p.ld;
  const long first = (long)run * s.run_chunks * kChunk, end = min(first + (long)s.run_chunks * kChunk, p.V);
  Cand *list = m.list[warp], *best = m.best[warp];
  int &count = m.count[warp];
  if (lane == 0) count = 0;
  if (tid == 0) m.bound = 0, m.total = 0;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;  // the warp's running maximum; this lane's sum against it
  int n = 0;                         // candidates in the list
  // if fewer than k values are above -inf, then of those at -inf only the run's first 2 k can be needed
  const long few = first + 2 * k;
  Chunk<T> next;
  if (first < end) next.load(logits, first, end);
  for (long at = first; at < end; at += kChunk) {
    const Chunk<T> c = next;
    if (at + kChunk < end) next.load(logits, at + kChunk, end);
    const int size = (int)min((long)kChunk, end - at);
    auto inside = [&](int i) { return c.place(i) < size; };
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = c.value(i);
    if (size < kChunk) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (!inside(i)) v[i] = -INFINITY;
    }
    constexpr int kPart = 8;  // values a part, whose largest is kept
    float most[kPer / kPart];
#pragma unroll
    for (int g = 0; g < kPer / kPart; ++g) {
      most[g] = v[g * kPart];
#pragma unroll
      for (int i = 1; i < kPart; ++i) most[g] = fmaxf(most[g], v[g * kPart + i]);
    }
    float mine = most[0];
#pragma unroll
    for (int g = 1; g < kPer / kPart; ++g) mine = fmaxf(mine, most[g]);
    bool odd = !(mine < INFINITY);  // an inf is there (a NaN shows in the sum)
    const float new_top = fmaxf(top, unordered(__reduce_max_sync(0xffffffffu, ordered(clean(mine)))));
    if (new_top > -INFINITY) {
      float2 part[2] = {both(0.f), both(0.f)};
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 d = __fmul2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), both(-new_top)), both(kLog2e));
        part[i >> 1 & 1] = __fadd2_rn(part[i >> 1 & 1], exp2_approx(d));
      }
      float all = (part[0].x + part[0].y) + (part[1].x + part[1].y);
      odd |= !(all < INFINITY);
      if (odd) {
        all = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = clean(v[i]), all += exp_under(v[i], new_top);
#pragma unroll
        for (int g = 0; g < kPer / kPart; ++g) most[g] = clean(most[g]);
      }
      sum = sum * exp_under(top, new_top) + all;
    } else {  // all -inf or NaN
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = -INFINITY;
#pragma unroll
      for (int g = 0; g < kPer / kPart; ++g) most[g] = -INFINITY;
    }
    mine = clean(mine);
    top = new_top;
    // one lane's reading for the whole warp: other warps raise the bound, and lanes that went apart above may read at
    // different times, which the shuffles below do not bear
    const uint32_t key = __shfl_sync(0xffffffffu, *(volatile uint32_t *)&m.bound, 0);
    float bound = key ? unordered(key) : -INFINITY;
    if (bound == -INFINITY) {  // one from these values alone: at least k reach it
      float x = mine;
      if (k > 32) {  // two of each lane: its second largest
        float largest = -INFINITY;
        x = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i) x = fmaxf(x, fminf(largest, v[i])), largest = fmaxf(largest, v[i]);
      }
      bound = __shfl_sync(0xffffffffu, warp_sort(x, lane), (k > 32 ? (k + 1) / 2 : k) - 1);
    }
    if (__any_sync(0xffffffffu, mine >= bound && (mine > -INFINITY || at < few))) {
#pragma unroll
      for (int g = 0; g < kPer / kPart; ++g) {
        if (!(most[g] >= bound)) continue;
#pragma unroll
        for (int j = 0; j < kPart; ++j) {
          const int i = g * kPart + j;
          if (v[i] >= bound && (v[i] > -INFINITY || (at + c.place(i) < few && inside(i)))) {
            const int o = atomicAdd(&count, 1);
            if (o < kCap) list[o] = Cand{ordered(v[i]), (uint32_t)at + c.place(i)};
          }
        }
      }
      __syncwarp();
      const int had = n;
      n = count;
      bool ranked = false;
      if (n > kCap) {
        // too many equal values: the k best of what the list had and of these, one after another
        Cand prev{0xffffffffu, 0u};
        for (n = 0; n < k; ++n) {
          Cand x{0u, 0xffffffffu};
          for (int i = lane; i < had; i += 32)
            if (before(prev, list[i]) && before(list[i], x)) x = list[i];
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const Cand y{ordered(v[i]), (uint32_t)at + c.place(i)};
            if (inside(i) && before(prev, y) && before(y, x)) x = y;
          }
          prev.key = __reduce_max_sync(0xffffffffu, x.key);
          prev.token = __reduce_min_sync(0xffffffffu, x.key == prev.key ? x.token : 0xffffffffu);
          if (prev.key == 0) break;
          if (lane == 0) best[n] = prev;
        }
        ranked = true;
      } else if (n >= k + 16) {
        rank_list(list, n, k, best, lane, 32);
        n = k;
        ranked = true;
      }
      if (ranked) {
        __syncwarp();
        for (int i = lane; i < n; i += 32) list[i] = best[i];
        if (lane == 0) {
          count = n;
          if (n == k) atomicMax(&m.bound, best[k - 1].key);
        }
        __syncwarp();
      }
    }
    if (at == first && at + kChunk < end) {  // the block's k-th best of the first chunk bounds the others
      rank_list(list, n, k, best, lane, 32);
      __syncthreads();
      place_candidates(m, k, [&](const Cand &x, int r) {
        if (r == k - 1) atomicMax(&m.bound, x.key);
      });
      __syncthreads();
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // not before: its blocks would take the others' places
  rank_list(list, n, k, best, lane, 32);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) m.top[warp] = top, m.sum[warp] = sum, atomicAdd(&m.total, min(n, k));
  __syncthreads();
  if (warp == 0) {
    const float t0 = lane < kWarps ? m.top[lane] : -INFINITY;
    const float t = unordered(__reduce_max_sync(0xffffffffu, ordered(t0)));
    float z = t0 > -INFINITY ? m.sum[lane] * exp_under(t0, t) : 0.f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) stat[0] = t, stat[1] = z;
  }
  place_candidates(m, k, [&](const Cand &x, int r) { out[r] = x; });
  if (tid < k && tid >= m.total) out[tid] = Cand{0u, 0u};  // fewer than k values in the run
}

// A continuation: its score in order as an unsigned number (0: none), its beam and token.
struct Scored {
  unsigned long long key;
  uint32_t beam, token;
};
__device__ __forceinline__ bool before(const Scored &a, const Scored &b) {
  return a.key > b.key ||
         (a.key == b.key && ((unsigned long long)a.beam << 32 | a.token) < ((unsigned long long)b.beam << 32 | b.token));
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double unordered(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}

// Candidates that are ranked by counting.  One group with many beams and runs lets more through the bound, and they are drawn
// one after another: 1 x 8 beams of 131072 with 16 continuations take 170 to 227 us (with 8, 57 us), 1 x 16 with 32 626 us,
// 1 x 64 with 64 4.8 ms.
constexpr int kJoinCap = 1024;

// Its time is that of its few 64-bit floating-point instructions one behind the other (this GPU issues one a
// warp in 64 cycles): a logarithm a row, three sums a candidate.
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const __grid_constant__ BeamProblem p, const __grid_constant__ BeamSplit s) {
  __shared__ double top[kMaxK], log_sum[kMaxK], score[kMaxK];
  __shared__ Scored list[kJoinCap], warp_best[kWarps];
  __shared__ uint32_t bound;  // of the keys' upper halves
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.k;
  const long g = blockIdx.x;
  const Cand *cands = reinterpret_cast<const Cand *>(s.cands) + g * p.W * s.runs * k;
  if (tid == 0) count = 0, bound = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the runs' kernel is through
  for (int w = warp; w < p.W; w += kWarps) {
    const float2 *st = reinterpret_cast<const float2 *>(s.stats) + (g * p.W + w) * s.runs;
    float t = -INFINITY, z = 0.f;
    for (int r = lane; r < s.runs; r += 32) t = fmaxf(t, st[r].x);
    t = unordered(__reduce_max_sync(0xffffffffu, ordered(t)));
    for (int r = lane; r < s.runs; r += 32)
      if (st[r].x > -INFINITY) z += st[r].y * exp_under(st[r].x, t);
    z = warp_sum(z);
    if (lane == 0) top[w] = t, log_sum[w] = log((double)z), score[w] = p.scores[g * p.W + w];
  }
  __syncthreads();
  const unsigned per_row = s.runs * k, all = p.W * per_row;
  auto scored = [&](unsigned i) {
    const Cand c = cands[i];
    if (c.key == 0) return Scored{0, ~0u, ~0u};
    const unsigned w = i / per_row;
    const double x = c.key == kMinusInf ? -INFINITY : score[w] + (((double)unordered(c.key) - top[w]) - log_sum[w]);
    return Scored{ordered(x), w, c.token};
  };
  // at least k continuations reach the best of the lists' last ones; the first kThreads continuations stay in registers
  const Scored mine = tid < all ? scored(tid) : Scored{0, ~0u, ~0u};
  for (unsigned i = tid; i < all; i += kThreads)
    if (i % k == k - 1) atomicMax(&bound, (uint32_t)((i < kThreads ? mine : scored(i)).key >> 32));
  __syncthreads();
  for (unsigned i = tid; i < all; i += kThreads) {
    const Scored x = i < kThreads ? mine : scored(i);
    if (x.key && (uint32_t)(x.key >> 32) >= bound) {
      const int n = atomicAdd(&count, 1);
      if (n < kJoinCap) list[n] = x;
    }
  }
  __syncthreads();
  const int n = count;
  auto put = [&](int r, const Scored &x) {
    const long o = g * k + r;
    p.out_scores[o] = (float)unordered(x.key), p.parents[o] = (int)x.beam, p.tokens[o] = (int)x.token;
  };
  if (n <= kJoinCap) {
    for (int i = tid; i < n; i += kThreads) {
      const Scored x = list[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += before(list[j], x);
      if (r < k) put(r, x);
    }
    return;
  }
  Scored prev{~0ull, 0, 0};
  for (int r = 0; r < k; ++r) {  // one after another, from the lists themselves
    Scored b{0, ~0u, ~0u};
    for (unsigned i = tid; i < all; i += kThreads) {
      const Scored x = scored(i);
      if (x.key && before(prev, x) && before(x, b)) b = x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Scored x{__shfl_xor_sync(0xffffffffu, b.key, o), __shfl_xor_sync(0xffffffffu, b.beam, o),
                     __shfl_xor_sync(0xffffffffu, b.token, o)};
      if (before(x, b)) b = x;
    }
    if (lane == 0) warp_best[warp] = b;
    __syncthreads();
    b = warp_best[0];
    for (int w = 1; w < kWarps; ++w)
      if (before(warp_best[w], b)) b = warp_best[w];
    prev = b;
    if (tid == 0) put(r, prev);
    __syncthreads();
  }
}

// A block takes a piece of one child's row, in every pool or (few beams) in one.  Which child copies from
// where to where every block works out from its group's parents, a thread a beam.
constexpr long kPiece = kReorderPiece;

__device__ __forceinline__ int nth_bit(unsigned long long x, int n) {
  for (; n > 0; --n) x &= x - 1;
  return x ? __ffsll(x) - 1 : -1;
}

__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const __grid_constant__ ReorderProblem p, int pieces, int spread) {
  __shared__ int parents[kMaxK], slots[kMaxK];
  __shared__ uint32_t masks[2][2];  // children that are the first of their parent; beams that have a child
  const int tid = threadIdx.x;
  long unit = blockIdx.x / pieces;
  const int piece = (int)(blockIdx.x - unit * pieces);
  const int only = (int)(unit % spread);
  unit /= spread;
  const int g = (int)(unit / p.W), j = (int)(unit - (long)g * p.W);
  if (tid < p.W) parents[tid] = p.parents[(long)g * p.W + tid], slots[tid] = p.slots[(long)g * p.W + tid];
  __syncthreads();
  if (tid < kMaxK) {
    bool first = tid < p.W && parents[tid] >= 0 && parents[tid] < p.W, has = false;
    for (int i = 0; i < p.W; ++i) {
      if (i < tid && first && parents[i] == parents[tid]) first = false;
      has |= parents[i] == tid;
    }
    const uint32_t f = __ballot_sync(0xffffffffu, first), c = __ballot_sync(0xffffffffu, has);
    if ((tid & 31) == 0) masks[0][tid >> 5] = f, masks[1][tid >> 5] = c;
  }
  __syncthreads();
  const unsigned long long firsts = (unsigned long long)masks[0][1] << 32 | masks[0][0];
  const unsigned long long parents_of = (unsigned long long)masks[1][1] << 32 | masks[1][0];
  const unsigned long long all = p.W == 64 ? ~0ull : (1ull << p.W) - 1, below = (1ull << j) - 1;
  const int parent = parents[j];
  const bool valid = parent >= 0 && parent < p.W, first = firsts >> j & 1;
  // as many beams have no child as there are children that are not the first of a beam
  const int to = slots[first ? parent : nth_bit(all & ~parents_of, __popcll(~firsts & below))];
  const bool lead = piece == 0 && only == 0 && p.first;
  if (lead && tid == 0) p.new_slots[(long)g * p.W + j] = to;
  if (first) return;
  const int from = valid ? slots[parent] : -1;
  bool bad = parent >= p.W || from >= p.n_slots || (from >= 0 && to >= p.n_slots);
  if (!bad && from >= 0 && to >= 0) {  // a slot that another beam of the batch has too is not written: it may be read
    // (all slots of the call, 4 G W bytes from L2 beside the piece's 32 KB: as much again at 1024 groups of 8)
    int times = 0;
    for (long i = tid; i < (long)p.G * p.W; i += kThreads) times += p.slots[i] == to;
    const int holders = __syncthreads_count(times > 0), more = __syncthreads_or(times > 1);
    bad = holders > 1 || more;
  }
  if (bad && lead && tid == 0) atomicOr(&g_beam_status, kStatusBadSlot);
  if (bad || from < 0 || to < 0) return;
  for (int l = only; l < p.pools; l += spread) {
    const long bytes = p.row_bytes[l], begin = piece * kPiece, end = min(begin + kPiece, bytes);
    const char *src = (const char *)p.pool[l] + from * bytes;
    char *dst = (char *)p.pool[l] + to * bytes;
    constexpr int kAhead = 8;
    for (long i = begin + tid * 16; i < end; i += kThreads * 16 * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i + u * kThreads * 16 < end) v[u] = __ldcs(reinterpret_cast<const uint4 *>(src + i + u * kThreads * 16));
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i + u * kThreads * 16 < end) __stcs(reinterpret_cast<uint4 *>(dst + i + u * kThreads * 16), v[u]);
    }
  }
}

cudaError_t launched(cudaError_t e, LaunchTimer &timer) {
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

// Runs of a row, of whole chunks: enough blocks for three an SM (each starts with its own bounds and ends with a join;
// six an SM took 80 us for 68 at 512 rows of 131072 in bf16).
BeamSplit beam_split(int G, int W, int k, long V) {
  BeamSplit s{};
  const long chunks = (V + kChunk - 1) / kChunk;
  const long rows = (long)G * W, want = 3L * std::max(1, device_info(-1).sm_count);
  const long runs = std::max(1L, std::min(chunks, (want + rows - 1) / rows));
  s.run_chunks = (int)((chunks + runs - 1) / runs);
  s.runs = (int)((chunks + s.run_chunks - 1) / s.run_chunks);
  s.bytes = (size_t)rows * s.runs * (k + 1) * 8;
  return s;
}

cudaError_t launch_beam_select(const BeamProblem &p) {
  BeamSplit s = beam_split(p.G, p.W, p.k, p.V);
  s.cands = p.ws;
  s.stats = (float *)((char *)p.ws + (size_t)p.G * p.W * s.runs * p.k * 8);
  const unsigned blocks = (unsigned)((long)p.G * p.W * s.runs);
  {
    LaunchTimer timer(kKBeamSelect, p.stream);
    if (p.dt == LA_F32)
      beam_rows_kernel<float><<<blocks, kThreads, 0, p.stream>>>(p, s);
    else
      beam_rows_kernel<__nv_bfloat16><<<blocks, kThreads, 0, p.stream>>>(p, s);
    const cudaError_t e = launched(cudaGetLastError(), timer);
    if (e != cudaSuccess) return e;
  }
  LaunchTimer timer(kKBeamSelect, p.stream);
  // launched early (programmatic dependent launch); it waits for the runs before it reads
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)p.G);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = p.stream;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, beam_join_kernel, p, s), timer);
}

// Few beams: a block for every pool of a child's row, so that one child's copies do not wait for each other.
cudaError_t launch_beam_reorder(const ReorderProblem &p) {
  long most = 1;
  for (int l = 0; l < p.pools; ++l) most = std::max(most, p.row_bytes[l]);
  const int pieces = (int)((most + kPiece - 1) / kPiece);
  const long units = (long)p.G * p.W * pieces;
  const int spread = units < 8L * std::max(1, device_info(-1).sm_count) ? std::max(1, p.pools) : 1;
  LaunchTimer timer(kKBeamReorder, p.stream);
  beam_reorder_kernel<<<(unsigned)(units * spread), kThreads, 0, p.stream>>>(p, pieces, spread);
  return launched(cudaGetLastError(), timer);
}

cudaError_t read_and_clear_beam_status(unsigned int *value) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_beam_status, sizeof(unsigned int));
  if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(g_beam_status, &zero, sizeof(unsigned int));
  return e;
}

}  // namespace la
