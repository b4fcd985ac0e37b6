// The next step of sequences over a paged cache, from the lengths on the device: which rows each one has, where
// they lie, and the pages for them (kv8_plan).
//
// With n = row0[b + 1] - row0[b] rows of the step before, of which take stay,
//   kept = kv_len - n + take,   need = max(0, ceil((kept + grow) / P) - held)   (0 without new rows)
// and prefix sums over the sequences of grow, need and the pages that ended sequences give back: the sums place every
// row, every new page (from the head of a ring of free pages) and every returned one (at its tail).
//
// What bounds it: nothing but latency.  A step of 64 windows touches some 6 KB, one with prompts some 300; a chain of
// dependent loads (offsets, sums over the block, search, page number) is all there is.  So the whole step is one launch:
// every CTA makes the same sums over all sequences (a thread for each, or for a few), then takes its share of the rows and pages,
// which are found by a binary search over the sums in shared memory.  Rows that land in a new page take its number from
// the ring, not from the table, so that nothing waits for another CTA.  What the sums are made of (offsets, lengths,
// pages held, the ring's state) is written by the last CTA to arrive, as the outputs may be the inputs' own buffers.
// Entries of the ring that are handed out and those that are filled are never the same: free pages and returned ones
// together are no more than its places.
//
// Measured: 64 windows of up to 8 5.5 us; 12 prompts of up to 2048 tokens among 1000 sequences, pages of 16, 9.0.  (A call from
// Python takes 9.6 of the host.)
#include "internal.h"
#include "kv8.cuh"

namespace w8a8 {
namespace plan {

constexpr int kMaxThreads = 1024;
constexpr int kRowsPerThread = 1;   // rows of the step's buffers for each thread: the grid's size (4: prompts among 1000 13.9 us, 1: 11.2)
constexpr int kMaxCtas = 128;
constexpr int kMost = (1 << 30) + 1;
__device__ __forceinline__ int plus(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kMost); }   // of numbers up to kMost
constexpr int kCounterWord = 16;    // of the workspace's header: arrivals of this call's CTAs, zero between calls

struct Params {
  const int *row0, *kv_len;
  int* table;
  int seqs, rows, max_tokens, width, shift;
  int* ring;
  const int* pool;
  int capacity;
  const int *held, *pinned, *take, *grow;
  int *row0_out, *kv_len_out, *held_out, *pool_out, *granted, *positions, *slots, *seq_of;
  uint32_t* status;
};

struct Seq {
  int kept, want, need, held, pinned, back;
};

// What sequence b asks for, before it is known whether it fits.  `report`: record indices that make no sense; such a
// sequence keeps its tokens and gets nothing.
__device__ __forceinline__ Seq load(const Params& p, int b, bool report) {
  const int r0 = p.row0[b], r1 = p.row0[b + 1], len = p.kv_len[b], take = p.take[b], grow = p.grow[b], held = p.held[b];
  const int pinned = p.pinned ? p.pinned[b] : 0;
  Seq s{max(len, 0), 0, 0, held, pinned, 0};
  const long long n = (long long)r1 - r0;
  bool ok = r0 >= 0 && n >= 0 && n <= len && held >= 0 && held <= p.width && pinned >= 0;
  if (ok && take < 0) {
    s.kept = 0;
    s.back = max(0, held - pinned);
    s.held = 0;
  } else if (ok) {
    const long long kept = len - n + take, pages = (kept + grow + (1 << p.shift) - 1) >> p.shift;
    ok = take <= n && grow >= 0 && grow <= p.max_tokens && pages <= p.width;
    if (ok) {
      s.kept = (int)kept;
      s.want = grow;
      s.need = grow > 0 ? max(0, (int)pages - held) : 0;
    }
  }
  if (!ok && report) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
  return s;
}

__global__ void __launch_bounds__(kMaxThreads) kv8_plan_kernel(const __grid_constant__ Params p) {
  __shared__ int warp_sm[3][32];
  __shared__ int rows_sm[kMaxThreads], need_sm[kMaxThreads], back_sm[kMaxThreads];   // sums before each thread's sequences
  __shared__ int fail_sm[32];
  __shared__ int total_sm[2];
  __shared__ int last_sm;
  pdl_trigger();
  pdl_wait();
  const int threads = blockDim.x, warps = threads >> 5, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.seqs + threads - 1) / threads;
  const int b0 = min(p.seqs, tid * per), b1 = min(p.seqs, b0 + per);
  const bool reporter = blockIdx.x == 0;
  int head = p.pool[0], free = p.pool[1];
  if (head < 0 || head >= p.capacity || free < 0 || free > p.capacity) {
    if (reporter && tid == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
    head = 0, free = 0;   // (none are handed out; what comes back fills the ring anew)
  }

  // ---------------------------------------------------------------- sums over the sequences
  // Of rows, pages and pages that come back, each held at kMost: more than any limit it is compared with.
  int mine[3] = {0, 0, 0}, before[3], all[3];
  for (int b = b0; b < b1; ++b) {
    const Seq s = load(p, b, reporter);
    mine[0] = plus(mine[0], s.want), mine[1] = plus(mine[1], s.need), mine[2] = plus(mine[2], s.back);
  }
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = plus(v, t);
    }
    return v;
  };
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int incl = scan(mine[i]), prev = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 31) warp_sm[i][warp] = incl;
    before[i] = lane > 0 ? prev : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int incl = scan(lane < warps ? warp_sm[i][lane] : 0), prev = __shfl_sync(0xffffffffu, incl, (warp + 31) & 31);
    before[i] = plus(before[i], warp > 0 ? prev : 0);
    all[i] = __shfl_sync(0xffffffffu, incl, 31);
  }
  // The first sequence that does not fit: from there on none gets rows.
  int fail = p.seqs;
  if (all[0] > p.rows || all[1] > free) {
    int r = before[0], n = before[1];
    for (int b = b0; b < b1 && fail == p.seqs; ++b) {
      const Seq s = load(p, b, false);
      r = plus(r, s.want), n = plus(n, s.need);
      if (r > p.rows || n > free) fail = b;
    }
    fail = __reduce_min_sync(0xffffffffu, fail);
    if (lane == 0) fail_sm[warp] = fail;
    __syncthreads();
    for (int w = 0; w < warps; ++w) fail = min(fail, fail_sm[w]);
    if (fail >= b0 && fail < b1) {
      r = before[0], n = before[1];
      for (int b = b0; b < fail; ++b) {
        const Seq s = load(p, b, false);
        r += s.want, n += s.need;
      }
      total_sm[0] = r, total_sm[1] = n;
    }
    __syncthreads();
    all[0] = total_sm[0], all[1] = total_sm[1];
  }
  const int rows = all[0], used = all[1];
  const int room = p.capacity - free;   // a ring that would hold more pages than places has been given one twice
  const int back = min(all[2], room);
  if (all[2] > room && reporter && tid == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
  rows_sm[tid] = min(before[0], rows);
  need_sm[tid] = min(before[1], used);
  back_sm[tid] = before[2];
  __syncthreads();

  // The sequence of place k in sums like `sums` (k below their total), and k's place within it.
  auto find = [&](const int* sums, int k, auto count, int& b, Seq& s) {
    int t = 0;
    for (int step = kMaxThreads / 2; step > 0; step >>= 1)
      if (t + step < threads && sums[t + step] <= k) t += step;
    k -= sums[t];
    b = t * per;
    s = load(p, b, false);
    while (k >= count(s) && b + 1 < p.seqs) {
      k -= count(s);
      s = load(p, ++b, false);
    }
    return k;
  };
  auto ring_at = [&](int i) {   // i at most the capacity
    const uint32_t at = (uint32_t)head + (uint32_t)i;
    return at < (uint32_t)p.capacity ? at : at - (uint32_t)p.capacity;
  };
  const int P = 1 << p.shift;
  const int first = blockIdx.x * threads + tid, stride = gridDim.x * threads;

  // ---------------------------------------------------------------- pages come back, pages go out
  for (int k = first; k < back; k += stride) {
    int b;
    Seq s;
    const int i = find(back_sm, k, [](const Seq& s) { return s.back; }, b, s);
    p.ring[ring_at(free + k)] = p.table[(size_t)b * p.width + s.pinned + i];
  }
  for (int k = first; k < used; k += stride) {
    int b;
    Seq s;
    const int i = find(need_sm, k, [](const Seq& s) { return s.need; }, b, s);
    p.table[(size_t)b * p.width + s.held + i] = p.ring[ring_at(k)];
  }
  // ---------------------------------------------------------------- rows
  if (p.positions || p.slots || p.seq_of) {
    for (int r = first; r < rows; r += stride) {
      int b;
      Seq s;
      const int i = find(rows_sm, r, [](const Seq& s) { return s.want; }, b, s);
      const int pos = s.kept + i, page = pos >> p.shift;
      if (p.positions) p.positions[r] = pos;
      if (p.seq_of) p.seq_of[r] = b;
      if (p.slots) {
        int id;
        if (page < s.held) {
          id = p.table[(size_t)b * p.width + page];
        } else {
          // A new page: its place in the ring is that of the pages before this sequence's.
          int at = need_sm[b / per];
          for (int c = b / per * per; c < b; ++c) at += load(p, c, false).need;
          id = p.ring[ring_at(at + page - s.held)];
        }
        p.slots[r] = (int)((uint32_t)id * (uint32_t)P + (uint32_t)(pos & (P - 1)));
      }
    }
  }
  // ---------------------------------------------------------------- what the sums are made of
  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      uint32_t* const counter = p.status + kCounterWord;
      const uint32_t old = atom_add_acq_rel_u32(counter, 1u);
      if (old >= gridDim.x) atomicOr(p.status, W8A8_DEV_COUNTER_CORRUPT);
      last_sm = old == gridDim.x - 1;
      if (last_sm) *counter = 0u;   // ready for the next call
    }
    __syncthreads();
    if (!last_sm) return;
  }
  // (The outputs may be the inputs' buffers.  A sequence reads two offsets: a thread has its first sequence before any
  // thread writes, and each further one before it writes the offset they share.)
  Seq s{};
  if (b0 < b1) s = load(p, b0, false);
  __syncthreads();
  int row = rows_sm[tid];
  for (int b = b0; b < b1; ++b) {
    const bool in = b < fail;
    const int got = in ? s.want : 0;
    p.kv_len_out[b] = s.kept + got;
    p.held_out[b] = s.held + (in ? s.need : 0);
    if (p.granted) p.granted[b] = got;
    if (b + 1 < b1) s = load(p, b + 1, false);
    row += got;
    p.row0_out[b + 1] = row;
  }
  if (tid == 0) {
    p.row0_out[0] = 0;
    p.pool_out[0] = (int)ring_at(used);
    p.pool_out[1] = free - used + back;
  }
}

}  // namespace plan
}  // namespace w8a8

using namespace w8a8;

extern "C" int kv8_plan(const kv8_step_t* step, int page_tokens, const kv8_pool_t* pool, const int32_t* held, const int32_t* pinned,
                        const int32_t* take, const int32_t* grow, const kv8_plan_t* out, void* ws, size_t ws_bytes, void* stream) {
  if (!step || !step->row0 || !step->kv_len || !step->page_table || step->seqs < 1 || step->seqs > 65535 || step->tokens < 0 ||
      step->tokens > (1 << 22) || step->max_tokens < 1 || step->max_tokens > (1 << 22) || step->table_width < 1)
    return W8A8_ERR_INVALID_ARG;
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128) return W8A8_ERR_UNSUPPORTED_SHAPE;
  if ((long long)step->table_width * page_tokens > (1ll << 30)) return W8A8_ERR_INVALID_ARG;
  if (!pool || !pool->ring || !pool->state || pool->capacity < 1 || pool->capacity > (1 << 30) || !held || !take || !grow || !out ||
      !out->row0 || !out->kv_len || !out->held || !out->pool_state)
    return W8A8_ERR_INVALID_ARG;
  const void* const words[] = {step->row0, step->kv_len, step->page_table, pool->ring, pool->state, held, pinned, take, grow, out->row0,
                               out->kv_len, out->held, out->pool_state, out->granted, out->positions, out->slots, out->seq_of};
  for (const void* w : words)
    if (!kv8_aligned(w, 4)) return W8A8_ERR_MISALIGNED;
  const int rc = kv8_check_ws(ws, ws_bytes, kWsHeaderBytes);
  if (rc != W8A8_OK) return rc;
  plan::Params p{};
  p.row0 = step->row0, p.kv_len = step->kv_len;
  p.table = const_cast<int*>(step->page_table);
  p.seqs = step->seqs, p.rows = step->tokens, p.max_tokens = step->max_tokens, p.width = step->table_width;
  p.shift = page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : 7;
  p.ring = pool->ring, p.pool = pool->state, p.capacity = pool->capacity;
  p.held = held, p.pinned = pinned, p.take = take, p.grow = grow;
  p.row0_out = out->row0, p.kv_len_out = out->kv_len, p.held_out = out->held, p.pool_out = out->pool_state;
  p.granted = out->granted, p.positions = out->positions, p.slots = out->slots, p.seq_of = out->seq_of;
  p.status = static_cast<uint32_t*>(ws);
  const int threads = step->seqs > 256 ? plan::kMaxThreads : 256, share = threads * plan::kRowsPerThread;
  const int ctas = step->tokens <= share ? 1 : step->tokens < share * plan::kMaxCtas ? (step->tokens + share - 1) / share : plan::kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, plan::kv8_plan_kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_plan");
}
