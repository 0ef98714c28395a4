// From request lengths to page tables, slots and offsets.  For sequence s with L_s cached positions and n_s new tokens:
//   rows [cu_s, cu_s + n_s) with cu the running sum of n;  row cu_s + i stands at position L_s + i;
//   P(L + n) - P(L) new pages, P(x) = ceil(x / page_size), taken from the top of a stack in the order of the sequences, so
//   the page of column c of s is stack[count - 1 - (pages of the sequences before + c - P(L_s))] whoever asks for it.
//
// Little work on the end of a chain of dependent loads: bound by latency.  Every workgroup therefore sums up the lengths for
// itself and no workgroup waits for another; it writes its rows (512, or 2048) from what it found.
// Offsets, lengths and the count are one workgroup's work: the same one for a call of one, an extra one for larger calls, and
// a launch ahead of the rows where they replace what is read or pages come back first; the rows are then found from them.
// 64 sequences' next tokens: 2.3 us on the GPU; 44514 rows of 211 sequences, of which 10 are over: 6.4 and 3.9 us.
#include "spa_attn.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kThreads = 512;
constexpr uint32_t kMost = 0x7FFFFFFFu;

struct Add {
  uint32_t most;                                       // sums stop here
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return min(a + b, most); }
  static constexpr int kNothing = 0;
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return (uint32_t)max((int)a, (int)b); }
  static constexpr int kNothing = -1;
};
template <int CTRL, int ROW_MASK, typename Op>
__device__ __forceinline__ uint32_t scan_step(uint32_t v, Op op) {
  return op(v, (uint32_t)__builtin_amdgcn_update_dpp(Op::kNothing, (int)v, CTRL, ROW_MASK, 0xF, false));
}
// What `op` makes of the lanes up to and with this one.
template <typename Op>
__device__ __forceinline__ uint32_t wave_scan_of(uint32_t v, Op op) {
  v = scan_step<0x111, 0xF>(v, op);    // within rows of 16
  v = scan_step<0x112, 0xF>(v, op);
  v = scan_step<0x114, 0xF>(v, op);
  v = scan_step<0x118, 0xF>(v, op);
  v = scan_step<0x142, 0xA>(v, op);    // the rows before
  return scan_step<0x143, 0xC>(v, op);
}
// What `op` makes of the threads before this one and, in `all`, of the whole workgroup of W waves.  The first half leaves each
// wave's result in s_wave; a barrier comes between.
template <int W>
__device__ __forceinline__ void scan_offer(uint32_t v, uint32_t (&s_wave)[W]) {
  if ((threadIdx.x & (kWave - 1)) == kWave - 1) s_wave[threadIdx.x / kWave] = v;
}
template <int W, typename Op>
__device__ __forceinline__ uint32_t scan_take(uint32_t v, Op op, const uint32_t (&s_wave)[W], uint32_t& all) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  uint32_t before = (uint32_t)Op::kNothing;
  all = (uint32_t)Op::kNothing;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == wave) before = all;
    all = op(all, s_wave[w]);
  }
  const uint32_t up = (uint32_t)__shfl_up((int)v, 1, kWave);
  return lane ? op(before, up) : before;
}

// A sequence as its rows see it: the row's position less its number; its number; the new pages before column 0, so that column
// c's is number pages + c; the columns that it had, and the page of the last of them.
struct Home { int shift, seq, pages, old, page; };

__device__ __forceinline__ int pages_of(const PlanArgs& a, int length) {
  return (int)a.page.div((uint32_t)(length + (int)a.page.d - 1));
}

// rows: this workgroup writes the rows from `first`, PER to a thread; commit: and, or, the offsets, lengths and count.  A thread
// holds PER sequences at a time.  count: the free pages.  AFTER: offsets, lengths and count are written already, and the state
// before is found from them: L + n and the running sums of n give L, count and all new pages what was free.
template <int THREADS, int PER, bool AFTER>
__device__ __forceinline__ void plan(const PlanArgs& a, int count, bool rows, bool commit, int first) {
  constexpr int kRows = THREADS * PER, W = THREADS / kWave;
  __shared__ uint32_t s_wave[4][W];
  __shared__ Home s_home[kRows + 1];                   // at a sequence's first row; the last: of the sequence that began before
  __shared__ int s_begins[kRows];
  const int tid = threadIdx.x, end = rows ? min(first + kRows, a.t) : 0;
  const int cap = a.max_pages * (int)a.page.d;
  if (rows)
#pragma unroll
    for (int i = 0; i < PER; ++i) s_begins[i * THREADS + tid] = -1;
  uint32_t done_rows = 0, done_pages = 0, done_keys = 0;       // of the sequences so far
  const Add fit{(uint32_t)a.t}, most{kMost};
  for (int base = 0; base < a.n_seqs; base += kRows) {
    int have[PER], fresh[PER], page[PER];
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = base + tid * PER + i;
      have[i] = fresh[i] = 0;
      if (s < a.n_seqs) {
        if constexpr (AFTER) {
          fresh[i] = a.cu_q[s + 1] - a.cu_q[s];
          have[i] = a.lens_out[s] - fresh[i];
        } else {
          const int length = a.lens[s], tokens = a.fresh[s], over = a.done ? a.done[s] : 0;
          have[i] = over ? 0 : min(max(length, 0), cap);
          fresh[i] = min(max(tokens, 0), a.t);
        }
      }
      sum = fit(sum, (uint32_t)fresh[i]);
    }
    // a page that is not full takes the first of the new rows
    if (rows)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int s = base + tid * PER + i, old = pages_of(a, have[i]);
        page[i] = -1;
        if (s < a.n_seqs && fresh[i] > 0 && old * (int)a.page.d > have[i]) page[i] = a.table[(size_t)s * a.max_pages + old - 1];
      }
    sum = wave_scan_of(sum, fit);
    scan_offer<W>(sum, s_wave[0]);
    __syncthreads();
    uint32_t all_rows, all_pages, all_keys;
    uint32_t at = fit(done_rows, scan_take<W>(sum, fit, s_wave[0], all_rows));
    uint32_t want = 0, keys = 0;
    int start[PER], need[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      start[i] = (int)at;
      const uint32_t to = fit(at, (uint32_t)fresh[i]);
      fresh[i] = (int)(to - at);                       // the rows end at t: what is past them is cut off
      at = to;
      need[i] = pages_of(a, min(have[i] + fresh[i], cap)) - pages_of(a, have[i]);
      want += (uint32_t)need[i];
      keys = most(keys, (uint32_t)(have[i] + fresh[i]));
    }
    want = wave_scan_of(want, most);
    keys = wave_scan_of(keys, most);
    scan_offer<W>(want, s_wave[1]);
    scan_offer<W>(keys, s_wave[2]);
    __syncthreads();
    uint32_t pages = done_pages + scan_take<W>(want, most, s_wave[1], all_pages);
    uint32_t key = most(done_keys, scan_take<W>(keys, most, s_wave[2], all_keys));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = base + tid * PER + i;
      const int old = pages_of(a, have[i]);
      if (rows && fresh[i] > 0 && start[i] < end && start[i] + fresh[i] > first) {
        const int local = start[i] < first ? kRows : start[i] - first;
        s_home[local] = Home{have[i] - start[i], s, (int)pages - old, old, page[i]};
        if (start[i] >= first) s_begins[local] = local;
      }
      if (commit && s < a.n_seqs) {
        key = most(key, (uint32_t)(have[i] + fresh[i]));
        a.cu_q[s + 1] = start[i] + fresh[i];
        a.cu_k[s + 1] = (int)key;
        a.lens_out[s] = have[i] + fresh[i];
      }
      pages += (uint32_t)need[i];
    }
    done_rows = fit(done_rows, all_rows);
    done_pages += all_pages;
    done_keys = most(done_keys, all_keys);
    __syncthreads();                                   // the homes are there; the scans' buffers may be written again
    if (!AFTER && !commit && (int)done_rows >= end) break;     // every row has its sequence
  }
  const int avail = AFTER ? count + (int)done_pages : min(max(count, 0), a.n_pages);
  if (commit && tid == 0) {
    a.cu_q[0] = a.cu_k[0] = 0;
    a.count_out[0] = max(avail - (int)min(done_pages, kMost), 0);
    a.count_out[1] = max((int)min(done_pages, kMost) - avail, 0);
  }
  if (!rows) return;
  if (a.n_seqs == 0) __syncthreads();                  // nothing has waited for s_begins yet
  int begins[PER];
  int best = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) best = begins[i] = max(best, s_begins[tid * PER + i]);
  const uint32_t upto = wave_scan_of((uint32_t)best, Max{});
  scan_offer<W>(upto, s_wave[3]);
  __syncthreads();
  uint32_t all;
  const int before = (int)scan_take<W>(upto, Max{}, s_wave[3], all);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = first + tid * PER + i;
    if (r >= end) break;
    const int at = max(before, begins[i]);
    int slot = -1, pos = 0;
    if (r < (int)done_rows) {
      const Home h = s_home[at < 0 ? kRows : at];
      pos = r + h.shift;
      if (pos < cap) {
        const int col = (int)a.page.div((uint32_t)pos), off = pos - col * (int)a.page.d;
        int pg = h.page;
        if (col >= h.old) {
          const int from = avail - 1 - (h.pages + col);
          pg = from >= 0 ? a.stack[from] : -1;
          if (pg >= a.n_pages) pg = -1;
          if (off == 0) a.table[(size_t)h.seq * a.max_pages + col] = max(pg, -1);
        }
        if (pg >= 0 && pg < a.n_pages) slot = pg * (int)a.page.d + off;
      }
    }
    a.slots[r] = slot;
    a.positions[r] = pos;
  }
}

// The pages of sequences that are over go back on the stack, in the order of the sequences and their columns.  One workgroup:
// it takes 512 sequences at a time, lists those that are over, counts their pages a wave to each, and copies them.  Returns what
// is free then.
__device__ __forceinline__ int release(const PlanArgs& a) {
  constexpr int kLook = 8, kWaves = kThreads / kWave;
  __shared__ uint32_t s_wave[2][kWaves];
  __shared__ int2 s_list[kThreads];                    // sequence, columns
  __shared__ int s_count[kThreads];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int cap = a.max_pages * (int)a.page.d;
  int count = min(max(a.count[0], 0), a.n_pages);
  for (int base = 0; base < a.n_seqs; base += kThreads) {
    const int s = base + tid;
    const int cols = s < a.n_seqs && a.done[s] ? pages_of(a, min(max(a.lens[s], 0), cap)) : 0;
    uint32_t listed, total;
    const uint32_t mine = wave_scan_of(cols > 0 ? 1u : 0u, Add{kMost});
    scan_offer<kWaves>(mine, s_wave[0]);
    __syncthreads();
    const uint32_t place = scan_take<kWaves>(mine, Add{kMost}, s_wave[0], listed);
    if (cols > 0) s_list[place] = make_int2(s, cols);
    s_count[tid] = 0;
    __syncthreads();
    // A wave's entries, every kWaves-th of the list, 64 columns at a time and kLook of these in flight, whosoever they are:
    // each(the entry's place in the list, a lane's page, whether it is one, whether the entry's columns end).  69 sequences of one
    // page that are over, of 345: 14.1 us a call, 21.3 with one entry at a time.
    auto walk = [&](auto each) {
      const int n_listed = __builtin_amdgcn_readfirstlane((int)listed);
      int at = __builtin_amdgcn_readfirstlane(wave), col = 0, seq = 0, cols = 0;
      auto open = [&] {
        if (at >= n_listed) return;
        seq = __builtin_amdgcn_readfirstlane(s_list[at].x);
        cols = __builtin_amdgcn_readfirstlane(s_list[at].y);
      };
      open();
      while (at < n_listed) {
        if (cols - col > kWave) {                      // a longer one: all in flight are its
          int pg[kLook];
          const int32_t* row = a.table + (size_t)seq * a.max_pages + col + lane;
#pragma unroll
          for (int u = 0; u < kLook; ++u) pg[u] = col + u * kWave + lane < cols ? row[u * kWave] : -1;
#pragma unroll
          for (int u = 0; u < kLook; ++u)
            if (col + u * kWave < cols) each(at, pg[u], pg[u] >= 0 && pg[u] < a.n_pages, col + (u + 1) * kWave >= cols);
          col += kWave * kLook;
          if (col >= cols) {
            at += kWaves;
            col = 0;
            open();
          }
          continue;
        }
        int pg[kLook], of[kLook];
        bool ends[kLook];
#pragma unroll
        for (int u = 0; u < kLook; ++u) {
          of[u] = at;
          pg[u] = -1;
          if (at < n_listed && col + lane < cols) pg[u] = a.table[(size_t)seq * a.max_pages + col + lane];
          col += kWave;
          ends[u] = at < n_listed && col >= cols;
          if (ends[u]) {
            at += kWaves;
            col = 0;
            open();
          }
        }
#pragma unroll
        for (int u = 0; u < kLook; ++u)
          if (of[u] < n_listed) each(of[u], pg[u], pg[u] >= 0 && pg[u] < a.n_pages, ends[u]);
      }
    };
    int n = 0;
    walk([&](int entry, int, bool ok, bool ends) {
      n += __popcll(__ballot(ok));
      if (!ends) return;
      if (lane == 0) s_count[entry] = n;
      n = 0;
    });
    __syncthreads();
    const uint32_t upto = wave_scan_of((uint32_t)s_count[tid], Add{kMost});
    scan_offer<kWaves>(upto, s_wave[1]);
    __syncthreads();
    const uint32_t before = scan_take<kWaves>(upto, Add{kMost}, s_wave[1], total);
    __syncthreads();
    s_count[tid] = (int)before;
    __syncthreads();
    int64_t to = -1;                                   // where the entry's next page goes
    walk([&](int entry, int pg, bool ok, bool ends) {
      if (to < 0) to = (int64_t)count + s_count[entry];
      const uint64_t there = __ballot(ok);
      const int64_t mine = to + __popcll(there & ((1ull << lane) - 1));
      if (ok && mine < a.n_pages) a.stack[mine] = pg;        // a stack holds every page once: it cannot be fuller
      to = ends ? -1 : to + __popcll(there);
    });
    count = (int)min((int64_t)count + total, (int64_t)a.n_pages);
    __syncthreads();
  }
  return count;
}

// mode: 0 rows and the rest in one workgroup; 1 rows, the last workgroup the rest; 2 the rest alone; 3 rows after it
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) k_kv_plan(PlanArgs a, int mode) {
  const int first = (int)blockIdx.x * THREADS * PER;
  if (mode == 3) {
    plan<THREADS, PER, true>(a, a.count_out[0] - a.count_out[1], true, false, first);
  } else {
    const bool rest = mode != 1 || blockIdx.x + 1 == gridDim.x;
    plan<THREADS, PER, false>(a, a.count[0], mode == 0 || !rest, rest, first);
  }
}
// Where sequences are over: mode 0 or 2 of the above behind their pages' return, in one workgroup.  64 sequences of which some are
// over: 6.1 us a call, 8.9 with a launch for the return; 211 with prompts of 45000 rows among them 11.2, 13.3.
template <int PER>
__global__ void __launch_bounds__(kThreads) k_kv_plan_done(PlanArgs a, int mode) {
  const int count = release(a);
  __syncthreads();                                     // what is on the stack now may be taken
  plan<kThreads, PER, false>(a, count, mode == 0, true, 0);
}

template <int THREADS, int PER>
hipError_t go(const PlanArgs& a, hipStream_t st) {
  const int blocks = (a.t + THREADS * PER - 1) / (THREADS * PER);
  auto run = [&](int grid, int mode) {
    hipLaunchKernelGGL((k_kv_plan<THREADS, PER>), dim3(grid), dim3(THREADS), 0, st, a, mode);
    return hipGetLastError();
  };
  if (a.done) {
    hipLaunchKernelGGL((k_kv_plan_done<PER>), dim3(1), dim3(kThreads), 0, st, a, blocks <= 1 ? 0 : 2);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    if (blocks <= 1) return run(1, 0);
    if (a.lens_out != a.lens && a.count_out != a.count) return run(blocks + 1, 1);
    if (hipError_t e = run(1, 2)) return e;
  }
  return blocks <= 1 ? hipSuccess : run(blocks, 3);
}

}  // namespace

hipError_t launch_kv_plan(PlanArgs a, hipStream_t st) {
  // As few rows to a workgroup as there are threads, if they also hold all sequences at once; one wave waits for nobody: 64
  // sequences take 2.5 us so, 5.4 with 512 threads of four.  More sequences: fewer workgroups that each sum them up.
  if (a.t <= kWave && a.n_seqs <= kWave && !a.done) return go<kWave, 1>(a, st);
  if (a.n_seqs <= kThreads) return go<kThreads, 1>(a, st);
  return go<kThreads, 4>(a, st);
}

}  // namespace spa
