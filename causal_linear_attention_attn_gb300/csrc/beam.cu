// Beam search over states: selection of the best continuations, and pools of states that follow them.
//
// Selection.  Of a group's W beams with scores s_w and logits l_{w,v} over V tokens, the k best by
//   s_w + l_{w,v} - log sum_v' e^{l_{w,v'}},
// in 64 bits (near a border the rounding of 32 bits would choose), ties to the lowest w V + v.  Within a beam the
// order is that of the logits, so the k best of each row are enough; HBM bounds it: the logits once.
//
// A block takes a run of one row in chunks of 8192 values held in registers, adds up its exponentials against a
// running maximum, and keeps candidates for the k best: each thread's largest value of the chunk, sorted across the
// warp's lanes, gives a value that at least k of the warp's values reach; the largest such bound of all warps and
// chunks lets a few dozen of the 8192 through.  Those are ranked by counting (every candidate against every other), not
// extracted one after another.  A second kernel, a block a group, joins the runs of a row and the rows of the
// group the same way in 64 bits.
//
// Reordering.  A beam's first child keeps the slot of its state in every pool; its other children get the
// slots of the group's childless beams, with a copy.  So the states move no more than they must, in place:
// what is read (kept slots) and what is written (freed ones) never meet.
#include <algorithm>

#include "internal.h"
#include "vec8.cuh"

namespace la {

__device__ unsigned int g_beam_status;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 32;                  // values a thread and chunk
constexpr int kChunk = kThreads * kPer;   // values a chunk
constexpr int kCap = 1024;                // candidates of a block
constexpr int kCompact = 256;             // more than these are ranked before the next chunk
constexpr int kMaxK = 64;

// NaN counts as -inf, inf as the largest finite number: infinite logits share the probability.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f); }
// e^(x - top), top finite
__device__ __forceinline__ float exp_under(float x, float top) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - top) * 1.44269504f));
  return y;
}
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
  // from place `at` behind base (aligned to 16 bytes): groups that begin before `row_end`, and nothing past `last`,
  // the end of the logits.
  __device__ __forceinline__ void load(const T *base, long at, const T *row_end, const T *last) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const T *p = base + at + ((long)j * kThreads + threadIdx.x) * kVec;
      a[j] = make_uint4(0u, 0u, 0u, 0u);
      if (p >= row_end) continue;
      if (p + kVec <= last) {
        a[j] = __ldcs(reinterpret_cast<const uint4 *>(p));
      } else {
        T *e = reinterpret_cast<T *>(&a[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (p + i < last) e[i] = p[i];
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
  Cand list[kCap], best[kMaxK];
  float bound[kWarps], top[kWarps], sum[kWarps];
  float threshold;
  int count;
};

// The k best of the list, in order, to best (key 0 behind the last); all threads.
__device__ __forceinline__ void rank_list(RowSmem &m, int n, int k) {
  if (threadIdx.x < kMaxK) m.best[threadIdx.x] = Cand{0u, 0u};
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Cand c = m.list[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += before(m.list[j], c);
    if (r < k) m.best[r] = c;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(const __grid_constant__ BeamProblem p, const __grid_constant__ BeamSplit s) {
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
  const T *base = (const T *)p.logits + row * p.ld, *last = (const T *)p.logits + ((long)p.G * p.W - 1) * p.ld + p.V;
  const int off = (int)((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
  base -= off;
  // places [off, off + V) behind base are the row's; this run's are whole chunks of them
  const long first = (long)run * s.run_chunks * kChunk, end = min(first + (long)s.run_chunks * kChunk, (long)off + p.V);
  const T *row_end = base + off + p.V;
  if (tid == 0) m.count = 0, m.threshold = -INFINITY;
  float top = -INFINITY, sum = 0.f;  // the warp's running maximum; this thread's sum against it
  const int share = k > 32 ? 2 : 1, each = (k + share - 1) / share;  // a bound takes `each` values of `share` warps
  // if fewer than k values are above -inf, then of those at -inf only the run's first 2 k can be needed
  const long few = max(first, (long)off) + 2 * k;
  Chunk<T> next;
  if (first < end) next.load(base, first, row_end, last);
  __syncthreads();
  for (long at = first; at < end; at += kChunk) {
    const Chunk<T> c = next;
    if (at + kChunk < end) next.load(base, at + kChunk, row_end, last);
    const int lo = (int)max(0L, off - at), hi = (int)min((long)kChunk, end - at);  // the row's places in this chunk
    const bool whole = lo == 0 && hi == kChunk;
    auto inside = [&](int i) { return whole || (c.place(i) >= lo && c.place(i) < hi); };
    auto value = [&](int i) { return inside(i) ? c.value(i) : -INFINITY; };
    float mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine = fmaxf(mine, value(i));
    mine = clean(mine);
    const float sorted = warp_sort(mine, lane);
    const float new_top = fmaxf(top, __shfl_sync(0xffffffffu, sorted, 0));
    if (new_top > -INFINITY) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kPer; ++i) part[i & 3] += exp_under(value(i), new_top);
      float all = (part[0] + part[1]) + (part[2] + part[3]);
      if (!(all < INFINITY)) {  // a NaN or inf among them
        all = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) all += exp_under(clean(value(i)), new_top);
      }
      sum = sum * exp_under(top, new_top) + all;
    }
    top = new_top;
    if (lane == each - 1) m.bound[warp] = sorted;
    __syncthreads();
    float b1 = -INFINITY, b2 = -INFINITY;  // the two largest of the warps' bounds
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float b = m.bound[w];
      b2 = fmaxf(b2, fminf(b1, b)), b1 = fmaxf(b1, b);
    }
    const float bound = fmaxf(m.threshold, share == 2 ? b2 : b1);
    const int had = m.count;
    __syncthreads();
    if (mine >= bound) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float v = clean(value(i));
        const long place = at + c.place(i);
        if (v >= bound && inside(i) && (v > -INFINITY || place < few)) {
          const int n = atomicAdd(&m.count, 1);
          if (n < kCap) m.list[n] = Cand{ordered(v), (uint32_t)(place - off)};
        }
      }
    }
    __syncthreads();
    int n = m.count;
    bool ranked = false;
    if (n > kCap) {
      // too many equal values: the k best of what the list had and of this chunk, one after another
      Cand prev{0xffffffffu, 0u};
      n = 0;
      for (; n < k; ++n) {
        Cand best{0u, 0xffffffffu};
        for (int i = tid; i < had; i += kThreads)
          if (before(prev, m.list[i]) && before(m.list[i], best)) best = m.list[i];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const Cand x{ordered(clean(value(i))), (uint32_t)(at + c.place(i) - off)};
          if (inside(i) && before(prev, x) && before(x, best)) best = x;
        }
        const uint32_t key = __reduce_max_sync(0xffffffffu, best.key);
        const uint32_t token = __reduce_min_sync(0xffffffffu, best.key == key ? best.token : 0xffffffffu);
        if (lane == 0) m.list[had + warp] = Cand{key, token};  // had <= kCompact
        __syncthreads();
        prev = m.list[had];
        for (int w = 1; w < kWarps; ++w)
          if (before(m.list[had + w], prev)) prev = m.list[had + w];
        if (tid == 0) m.best[n] = prev;
        __syncthreads();
        if (prev.key == 0) break;
      }
      ranked = true;
    } else if (n > kCompact) {
      rank_list(m, n, k);
      n = min(n, k);
      ranked = true;
    }
    if (ranked && tid < n) m.list[tid] = m.best[tid];
    __syncthreads();
    if (tid == 0) {
      m.count = n;
      m.threshold = ranked && n == k ? fmaxf(bound, unordered(m.list[n - 1].key)) : bound;
    }
    __syncthreads();
  }
  rank_list(m, m.count, k);
  if (tid < k) out[tid] = m.best[tid];
  // the row's maximum and sum over the block
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) m.top[warp] = top, m.sum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    float t = m.top[0], z = 0.f;
    for (int w = 1; w < kWarps; ++w) t = fmaxf(t, m.top[w]);
    for (int w = 0; w < kWarps; ++w)
      if (m.top[w] > -INFINITY) z += m.sum[w] * exp_under(m.top[w], t);
    stat[0] = t, stat[1] = z;
  }
}

struct Scored {
  double score;
  long flat;  // w V + v, or -1: none
};
__device__ __forceinline__ bool before(const Scored &a, const Scored &b) {
  if (a.flat < 0 || b.flat < 0) return b.flat < 0 && a.flat >= 0;
  return a.score > b.score || (a.score == b.score && a.flat < b.flat);
}

constexpr int kJoinCap = 1024;

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const __grid_constant__ BeamProblem p, const __grid_constant__ BeamSplit s) {
  __shared__ double top[kMaxK], log_sum[kMaxK];
  __shared__ Scored list[kJoinCap], warp_best[kWarps];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.k;
  const long g = blockIdx.x;
  const Cand *cands = reinterpret_cast<const Cand *>(s.cands) + g * p.W * s.runs * k;
  for (int w = warp; w < p.W; w += kWarps) {
    const float *st = s.stats + (g * p.W + w) * s.runs * 2;
    float t = -INFINITY;
    for (int r = lane; r < s.runs; r += 32) t = fmaxf(t, st[2 * r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    double z = 0.;
    for (int r = lane; r < s.runs; r += 32)
      if (st[2 * r] > -INFINITY) z += (double)st[2 * r + 1] * (st[2 * r] == t ? 1. : exp((double)st[2 * r] - (double)t));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) top[w] = t, log_sum[w] = log(z);
  }
  if (tid == 0) count = 0;
  __syncthreads();
  const int lists = p.W * s.runs;
  auto scored = [&](int l, int i) {
    const Cand c = cands[(long)l * k + i];
    if (c.key == 0) return Scored{0., -1};
    const int w = l / s.runs;
    const double score = c.key == kMinusInf ? -INFINITY
                                            : (double)p.scores[g * p.W + w] + (((double)unordered(c.key) - top[w]) - log_sum[w]);
    return Scored{score, (long)w * p.V + c.token};
  };
  auto block_best = [&](Scored b) {  // the first in order of all threads'
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Scored x{__shfl_xor_sync(0xffffffffu, b.score, o), __shfl_xor_sync(0xffffffffu, b.flat, o)};
      if (before(x, b)) b = x;
    }
    __syncthreads();
    if (lane == 0) warp_best[warp] = b;
    __syncthreads();
    b = warp_best[0];
    for (int w = 1; w < kWarps; ++w)
      if (before(warp_best[w], b)) b = warp_best[w];
    return b;
  };
  // no list's last candidate may be beaten by a chosen one's successor: what comes before the best of them is enough
  Scored bound{0., -1};
  for (int l = tid; l < lists; l += kThreads) {
    const Scored x = scored(l, k - 1);
    if (before(x, bound)) bound = x;
  }
  bound = block_best(bound);
  for (int i = tid; i < lists * k; i += kThreads) {
    const Scored x = scored(i / k, i % k);
    if (x.flat >= 0 && !before(bound, x)) {
      const int n = atomicAdd(&count, 1);
      if (n < kJoinCap) list[n] = x;
    }
  }
  __syncthreads();
  const int n = count;
  auto put = [&](int r, const Scored &x) {
    const long o = g * k + r;
    const int w = (int)(x.flat / p.V);
    p.out_scores[o] = (float)x.score, p.parents[o] = w, p.tokens[o] = (int)(x.flat - (long)w * p.V);
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
  Scored prev{INFINITY, -2};
  for (int r = 0; r < k; ++r) {  // one after another, from the lists themselves
    Scored b{0., -1};
    for (int i = tid; i < lists * k; i += kThreads) {
      const Scored x = scored(i / k, i % k);
      if ((prev.flat == -2 || before(prev, x)) && before(x, b)) b = x;
    }
    prev = block_best(b);
    if (tid == 0) put(r, prev);
  }
}

// A block takes a piece of one child's row, in every pool or (few beams) in one.  Which child copies from
// where to where every block works out from its group's parents, a thread a beam.
constexpr long kPiece = 32768;  // bytes

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

// Runs of a row: enough blocks for four an SM, of whole chunks (a row may begin up to 16 bytes behind its first chunk's
// start).
BeamSplit beam_split(int G, int W, int k, long V, la_dtype dt) {
  BeamSplit s{};
  const long chunks = (V + 16 / (dt == LA_F32 ? 4 : 2) - 1 + kChunk - 1) / kChunk;
  const long rows = (long)G * W, want = 4L * std::max(1, device_info(-1).sm_count);
  const long runs = std::max(1L, std::min(chunks, (want + rows - 1) / rows));
  s.run_chunks = (int)((chunks + runs - 1) / runs);
  s.runs = (int)((chunks + s.run_chunks - 1) / s.run_chunks);
  s.bytes = (size_t)rows * s.runs * (k + 1) * 8;
  return s;
}

cudaError_t launch_beam_select(const BeamProblem &p) {
  BeamSplit s = beam_split(p.G, p.W, p.k, p.V, p.dt);
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
  beam_join_kernel<<<(unsigned)p.G, kThreads, 0, p.stream>>>(p, s);
  return launched(cudaGetLastError(), timer);
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
