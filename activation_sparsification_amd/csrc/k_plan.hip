// From request lengths to page tables, slots and offsets.  For sequence s with L_s cached positions and n_s new tokens:
//   rows [cu_s, cu_s + n_s) with cu the running sum of n;  row cu_s + i stands at position L_s + i;
//   P(L + n) - P(L) new pages, P(x) = ceil(x / page_size), taken from the top of a stack in the order of the sequences, so
//   the page of column c of s is stack[count - 1 - (pages of the sequences before + c - P(L_s))] whoever asks for it.
//
// Little work on the end of a chain of dependent loads: bound by latency.  Every workgroup therefore sums up the lengths for
// itself (a thread holds four sequences) and no workgroup waits for another; it writes its 2048 rows from what it found.
// Offsets, lengths and the count are one workgroup's work: the same one for a call of one, an extra one for larger calls,
// and a launch of its own where they replace the values that the others read.
#include "spa_attn.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kThreads = 512, kPer = 4;                // sequences, and rows, of a thread
constexpr int kRows = kThreads * kPer;                 // of a workgroup
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
// What `op` makes of the threads before this one and, in `all`, of the whole workgroup.
template <typename Op>
__device__ __forceinline__ uint32_t scan_before(uint32_t v, Op op, uint32_t (&s_wave)[kThreads / kWave], uint32_t& all) {
  v = scan_step<0x111, 0xF>(v, op);    // within rows of 16
  v = scan_step<0x112, 0xF>(v, op);
  v = scan_step<0x114, 0xF>(v, op);
  v = scan_step<0x118, 0xF>(v, op);
  v = scan_step<0x142, 0xA>(v, op);    // the rows before
  v = scan_step<0x143, 0xC>(v, op);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  if (lane == kWave - 1) s_wave[wave] = v;
  __syncthreads();
  uint32_t before = (uint32_t)Op::kNothing;
  all = (uint32_t)Op::kNothing;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w == wave) before = all;
    all = op(all, s_wave[w]);
  }
  const uint32_t up = (uint32_t)__shfl_up((int)v, 1, kWave);
  return lane ? op(before, up) : before;
}

// A sequence as its rows see it: the row's position less its number; its number; the new pages before column 0, so that column
// c's is number pages + c; the columns that it had.
struct Home { int shift, seq, pages, old; };

__device__ __forceinline__ int pages_of(const PlanArgs& a, int length) {
  return (int)a.page.div((uint32_t)(length + (int)a.page.d - 1));
}

// rows: this workgroup writes rows; commit: and, or, the offsets, lengths and count.
__device__ __forceinline__ void plan(const PlanArgs& a, bool rows, bool commit, int first) {
  __shared__ uint32_t s_wave[3][kThreads / kWave];
  __shared__ Home s_home[kRows + 1];                   // at a sequence's first row; the last: of the sequence that began before
  __shared__ int s_begins[kRows];
  const int tid = threadIdx.x, end = rows ? min(first + kRows, a.t) : 0;
  const int cap = a.max_pages * (int)a.page.d;
  const int avail = min(max(a.count[0], 0), a.n_pages);
  if (rows)
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_begins[i * kThreads + tid] = -1;
  uint32_t done_rows = 0, done_pages = 0, done_keys = 0;       // of the sequences so far
  if (rows && tid == 0) s_home[kRows].seq = -1;
  for (int base = 0; base < a.n_seqs; base += kThreads * kPer) {
    int have[kPer], fresh[kPer];
    uint32_t sum = 0;
    const Add fit{(uint32_t)a.t};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = base + tid * kPer + i;
      have[i] = fresh[i] = 0;
      if (s < a.n_seqs) {
        have[i] = a.done && a.done[s] ? 0 : min(max(a.lens[s], 0), cap);
        fresh[i] = min(max(a.fresh[s], 0), a.t);
      }
      sum = fit(sum, (uint32_t)fresh[i]);
    }
    uint32_t all_rows, all_pages, all_keys = 0;
    // (a third buffer in turn would do for the barriers; three are simpler: each is written again only after the others' barriers)
    uint32_t row = fit(done_rows, scan_before(sum, fit, s_wave[0], all_rows));
    uint32_t want = 0, keys = 0;
    const Add most{kMost};
    int start[kPer], need[kPer];
    uint32_t at = row;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      start[i] = (int)at;
      const uint32_t to = fit(at, (uint32_t)fresh[i]);
      fresh[i] = (int)(to - at);                       // the rows end at t: what is past them is cut off
      at = to;
      need[i] = pages_of(a, min(have[i] + fresh[i], cap)) - pages_of(a, have[i]);
      want += (uint32_t)need[i];
      keys = most(keys, (uint32_t)(have[i] + fresh[i]));
    }
    uint32_t page = done_pages + scan_before(want, most, s_wave[1], all_pages);
    uint32_t key = commit ? most(done_keys, scan_before(keys, most, s_wave[2], all_keys)) : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = base + tid * kPer + i;
      const int old = pages_of(a, have[i]);
      if (rows && fresh[i] > 0 && start[i] < end && start[i] + fresh[i] > first) {
        const int local = start[i] < first ? kRows : start[i] - first;
        s_home[local] = Home{have[i] - start[i], s, (int)page - old, old};
        if (start[i] >= first) s_begins[local] = local;
      }
      if (commit && s < a.n_seqs) {
        key = most(key, (uint32_t)(have[i] + fresh[i]));
        a.cu_q[s + 1] = start[i] + fresh[i];
        a.cu_k[s + 1] = (int)key;
        a.lens_out[s] = have[i] + fresh[i];
      }
      page += (uint32_t)need[i];
    }
    done_rows = fit(done_rows, all_rows);
    done_pages += all_pages;
    done_keys = most(done_keys, all_keys);
    __syncthreads();                                   // the scans' buffers and, after the last, the homes
    if (!commit && (int)done_rows >= end) break;       // every row has its sequence
  }
  if (commit && tid == 0) {
    a.cu_q[0] = a.cu_k[0] = 0;
    a.count_out[0] = max(avail - (int)min(done_pages, kMost), 0);
    a.count_out[1] = max((int)min(done_pages, kMost) - avail, 0);
  }
  if (!rows) return;
  __syncthreads();
  int begins[kPer];
  int best = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) best = begins[i] = max(best, s_begins[tid * kPer + i]);
  uint32_t all;
  const int before = (int)scan_before((uint32_t)best, Max{}, s_wave[0], all);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = first + tid * kPer + i;
    if (r >= end) break;
    const int at = max(before, begins[i]);
    int slot = -1, pos = 0;
    if (r < (int)done_rows) {
      const Home h = s_home[at < 0 ? kRows : at];
      pos = r + h.shift;
      if (pos < cap) {
        const int col = (int)a.page.div((uint32_t)pos), off = pos - col * (int)a.page.d;
        int pg;
        if (col < h.old) {
          pg = a.table[(size_t)h.seq * a.max_pages + col];
        } else {
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

// mode: 0 rows and the rest in one workgroup; 1 rows, the last workgroup the rest; 2 rows alone; 3 the rest alone
__global__ void __launch_bounds__(kThreads) k_kv_plan(PlanArgs a, int mode) {
  const bool last = blockIdx.x + 1 == gridDim.x;
  const bool rows = mode == 0 || mode == 2 || (mode == 1 && !last);
  plan(a, rows, mode == 0 || mode == 3 || (mode == 1 && last), (int)blockIdx.x * kRows);
}

// The pages of sequences that are over go back on the stack, in the order of the sequences and their columns.  One workgroup:
// it takes 512 sequences at a time, lists those that are over, counts their pages a wave to each, and copies them.
__global__ void __launch_bounds__(kThreads) k_kv_release(PlanArgs a) {
  constexpr int kLook = 8;                             // entries of a lane in flight
  __shared__ uint32_t s_wave[2][kThreads / kWave];
  __shared__ int2 s_list[kThreads];                    // sequence, columns
  __shared__ int s_count[kThreads];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int cap = a.max_pages * (int)a.page.d;
  int count = min(max(a.count[0], 0), a.n_pages);
  for (int base = 0; base < a.n_seqs; base += kThreads) {
    const int s = base + tid;
    const int cols = s < a.n_seqs && a.done[s] ? pages_of(a, min(max(a.lens[s], 0), cap)) : 0;
    uint32_t listed, total;
    const uint32_t place = scan_before(cols > 0 ? 1u : 0u, Add{kMost}, s_wave[0], listed);
    if (cols > 0) s_list[place] = make_int2(s, cols);
    s_count[tid] = 0;
    __syncthreads();
    auto walk = [&](int2 e, auto each) {               // each(entry's page, whether it is one)
      const int32_t* row = a.table + (size_t)e.x * a.max_pages;
      for (int c = lane; c - lane < e.y; c += kLook * kWave) {
        int pg[kLook];
#pragma unroll
        for (int u = 0; u < kLook; ++u) pg[u] = c + u * kWave < e.y ? row[c + u * kWave] : -1;
#pragma unroll
        for (int u = 0; u < kLook; ++u) each(pg[u], pg[u] >= 0 && pg[u] < a.n_pages);
      }
    };
    for (int i = wave; i < (int)listed; i += kThreads / kWave) {
      int n = 0;
      walk(s_list[i], [&](int, bool ok) { n += __popcll(__ballot(ok)); });
      if (lane == 0) s_count[i] = n;
    }
    __syncthreads();
    const uint32_t before = scan_before((uint32_t)s_count[tid], Add{kMost}, s_wave[1], total);
    __syncthreads();
    s_count[tid] = (int)before;
    __syncthreads();
    for (int i = wave; i < (int)listed; i += kThreads / kWave) {
      int64_t to = (int64_t)count + s_count[i];
      walk(s_list[i], [&](int pg, bool ok) {
        const uint64_t there = __ballot(ok);
        const int64_t mine = to + __popcll(there & ((1ull << lane) - 1));
        if (ok && mine < a.n_pages) a.stack[mine] = pg;      // a stack holds every page once: it cannot be fuller
        to += __popcll(there);
      });
    }
    count = (int)min((int64_t)count + total, (int64_t)a.n_pages);
    __syncthreads();
  }
  if (tid == 0) a.count_out[0] = count;
}

}  // namespace

hipError_t launch_kv_plan(PlanArgs a, hipStream_t st) {
  bool replaces = a.lens_out == a.lens || a.count_out == a.count;
  if (a.done) {
    hipLaunchKernelGGL(k_kv_release, dim3(1), dim3(kThreads), 0, st, a);
    if (hipError_t e = hipGetLastError()) return e;
    a.count = a.count_out;
    replaces = true;
  }
  const int blocks = (a.t + kRows - 1) / kRows;
  if (blocks <= 1) {
    hipLaunchKernelGGL(k_kv_plan, dim3(1), dim3(kThreads), 0, st, a, 0);
  } else if (!replaces) {
    hipLaunchKernelGGL(k_kv_plan, dim3(blocks + 1), dim3(kThreads), 0, st, a, 1);
  } else {
    hipLaunchKernelGGL(k_kv_plan, dim3(blocks), dim3(kThreads), 0, st, a, 2);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL(k_kv_plan, dim3(1), dim3(kThreads), 0, st, a, 3);
  }
  return hipGetLastError();
}

}  // namespace spa
