// kv_attn.cuh -- what the attention kernels over the paged cache share: the
// arguments, the division of the work among CTAs, partial results.  Internal
// to the library.
//
// Work.  The query rows of one sequence and one key/value head are the pairs
// (new token i, query head g of the group), row i * G + g, so that a row tile
// reads each key once for all heads of the group.  A row tile of one sequence
// is an entry; its cost is its number of KV tiles (kTile keys; at least one,
// so that rows which see nothing are written too), and before them lead_units
// for what an entry takes besides.  The entries' costs in a row, once for each key/value head, are the units; worker c (a CTA of the
// chunk kernel, a warp of the step kernel) takes the units [c * share, (c + 1) *
// share), whatever sequences and heads they fall in.  An entry that lies in
// several workers' shares leaves partial results (FP32 O, row maxima and sums)
// in the workspace, which the combine kernel joins in the workers' order: the
// split depends on the lengths alone, so repeated calls give the same bits.
#pragma once

#include "kv.cuh"

namespace sagefp4 {

constexpr int kTile = 128;       // keys of a KV tile
constexpr int kChunkRows = 256;  // query rows of an entry: two row tiles of 128
constexpr int kMaxSms = 160;     // the workspace's partial results are for this many at most

struct AttnArgs {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  sage_kv_rows qr, orow;
  int T, Hq, G;       // packed rows, query heads, query heads per key/value head
  int causal, window;
  float scale_log2;   // softmax scale * log2(e)
};

// One row tile of one sequence: rows from row0 of its G * (new tokens), `tiles`
// KV tiles from t0 on (t0 = -1: no key is seen; one for the count).
struct __align__(16) PlanEntry {
  int q0, nq, len, b;   // first packed row, new tokens, cached tokens, sequence
  int row0, t0, tiles, pad;
};

struct PlanHead {
  long long units;  // of one key/value head
  int entries;
  int pad;
};

// The device's plan, partial results and error state of one call.
struct AttnWork {
  PlanHead* head;
  PlanEntry* entry;    // [capacity]
  long long* cum;      // [capacity]: units of the entries before
  float* part_o;       // slots [2 * workers]: [D / 4][rows][4] (chunk), [rows][D] (step)
  float2* part_ml;     // [2 * workers][rows]: row maximum (log2 units), sum
  int2* open;          // [workers] (chunk): entry and head that a share begins and does not end (-1: none)
  int capacity, workers, lead_units;
  long long min_share;
  uint64_t wait_ns;
  int withhold;        // (chunk, failure test) the first CTA never announces its first scores
};

__device__ __forceinline__ long long share_of(long long units, int workers, long long min_share) {
  const long long s = (units + workers - 1) / workers;
  return s > min_share ? s : min_share;
}

// Keys that the row of new token i sees: [lo, hi).
__device__ __forceinline__ int2 key_range(const AttnArgs& a, int len, int nq, int i) {
  const int pos = len - nq + i;
  const int hi = a.causal ? min(len, pos + 1) : len;
  // (pos may be negative and the window any int: no difference of the two below 0)
  const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
  return int2{lo, hi};
}

// The first key that an entry's rows see, down to the 16 whose page is looked
// up at once: pages before it may be gone.
__device__ __forceinline__ int first_key(const AttnArgs& a, int len, int nq, int row0) {
  return key_range(a, len, nq, row0 / a.G).x & ~15;
}

// KV tiles of the rows [row0, row1): {first, end}.
__device__ __forceinline__ int2 tile_range(const AttnArgs& a, int len, int nq, int row0, int row1) {
  const int hi = key_range(a, len, nq, (row1 - 1) / a.G).y;
  const int lo = key_range(a, len, nq, row0 / a.G).x;
  if (hi <= lo) return int2{0, 0};
  return int2{lo / kTile, (hi + kTile - 1) / kTile};
}

// The entry of the rows row0 .. (`rows` at most) of sequence b's new tokens.
__device__ __forceinline__ PlanEntry make_entry(const AttnArgs& a, int rows, int q0, int nq, int len, int b, int row0) {
  const int2 t = tile_range(a, len, nq, row0, min(row0 + rows, nq * a.G));
  return PlanEntry{q0, nq, len, b, row0, t.y > t.x ? t.x : -1, t.y > t.x ? t.y - t.x : 1, 0};
}

// First unit of a worker, before the border's move.
__device__ __forceinline__ long long first_unit(const AttnWork& w, int heads, int worker) {
  const long long total = w.head->units * heads, u = share_of(total, w.workers, w.min_share) * worker;
  return u < total ? u : total;
}

// Entry that holds unit r of a head: the last with cum <= r.
__device__ __forceinline__ int entry_at(const AttnWork& w, long long r) {
  int lo = 0, hi = w.head->entries;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (w.cum[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// A worker's walk over its units, one entry (or a part of one) after the
// other.  Every thread of every role walks alike.
struct Walk {
  int left, off;  // units left; of the next entry, those before the worker's share
  int j, h;       // next entry, its key/value head
  // the current piece: entry j - 1, head h, KV tiles t .. t + tiles - 1 (none
  // for rows that see nothing); first / last: it begins / ends the entry
  int t, tiles;
  bool first, last;

  __device__ __forceinline__ Walk(const AttnWork& w, int heads, int worker) {
    const long long units = w.head->units, total = units * heads;
    left = off = j = h = 0;
    long long u = first_unit(w, heads, worker), end = first_unit(w, heads, worker + 1);
    if (u == end) return;
    if (end < total) {
      const long long r = end % units;
      const int past = static_cast<int>(r - w.cum[entry_at(w, r)]);
      if (past <= w.lead_units) end -= past;
    }
    h = static_cast<int>(u / units);
    const long long r = u - units * h;
    j = entry_at(w, r);
    off = static_cast<int>(r - w.cum[j]);
    if (off <= w.lead_units) {
      u -= off;
      off = 0;
    }
    left = static_cast<int>(end - u);
  }

  __device__ __forceinline__ bool next(const AttnWork& w) {
    if (left == 0) return false;
    if (j == w.head->entries) {
      j = 0;
      h++;
    }
    const int cost = w.entry[j].tiles + w.lead_units, t0 = w.entry[j].t0;
    const int n = cost - off < left ? cost - off : left;
    const int from = off > 0 ? off - w.lead_units : 0;
    t = t0 + from;
    tiles = t0 < 0 ? 0 : off + n - w.lead_units - from;
    first = off == 0;
    last = off + n == cost;
    off = 0;
    left -= n;
    j++;
    return true;
  }

  __device__ __forceinline__ const PlanEntry& entry(const AttnWork& w) const { return w.entry[j - 1]; }
};

// Launch a kernel that calls griddep_wait() before it reads what the kernel
// queued before it writes: it may be resident by then.
template <typename... A, typename... B>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, int shared, cudaStream_t st, B&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<B&&>(args)...);
}

// Allow a kernel its dynamic shared memory, once for each device.
template <auto kKernel>
cudaError_t set_shared_once(int bytes) {
  static std::atomic<bool> done[64];  // racing threads set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

cudaError_t launch_attn_chunk(const KvView& c, const AttnArgs& a, const AttnWork& w, int D, int format, cudaStream_t st);
// rows: of an entry, 8 or 16.
cudaError_t launch_attn_step(const KvView& c, const AttnArgs& a, const AttnWork& w, int rows, int D, int format,
                             cudaStream_t st);

}  // namespace sagefp4
