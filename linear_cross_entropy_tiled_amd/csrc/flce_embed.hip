// Token embedding, out_i = scale weight[id_i], and its gradient
//   grad_weight_v = scale sum over the tokens i with id_i = v of grad_i.
//
// The gradient brings tokens of the same id together (in their order, so that results do
// not depend on timing), then sums each run of equal ids in
// fp32 and rounds it once.  Runs are summed by chunks of sorted tokens, not by rows: a
// frequent token's run of thousands is spread over many workgroups.  The part of a run
// that reaches over a chunk's edge is left in fp32 and a second kernel adds the parts.
//
// What bounds it is memory, and of the whole gradient mostly its zeros.  N = 8192, H = 4096,
// V = 128256, bf16, Zipf's ids: forward 29 us in a training step (22 to 31; its 112 MB at 3.9
// TB/s), zeros and sort 165 us (1.05 GB at 6.4 TB/s, where a plain fill reaches 6.9), runs 36,
// joins 10.
#include "flce_device.h"
#include "flce_embed.h"

namespace flce {

struct EmbedArgs {
  const void* ids;
  int ids_i32;
  int64_t n, v, ignore_index;
  int h;
  float scale;
  const void* weight;
  void* out;
};

// The id of token i as a row of the weight, or v for a token that is none.
__device__ __forceinline__ uint32_t row_of(const EmbedArgs& a, int64_t i) {
  const int64_t t = load_target(a.ids, i, a.ids_i32);
  return (uint32_t)(t != a.ignore_index && t >= 0 && t < a.v ? t : a.v);
}

// ---------------------------------------------------------------------------
// Forward: one wave a token, VEC elements (16 bytes, or 1 where rows are not aligned) a lane,
// kPieces of them in flight
// ---------------------------------------------------------------------------
template <typename T, int VEC> __global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedArgs a) {
  typedef T V __attribute__((ext_vector_type(VEC)));
  constexpr int kPieces = 8;
  const int lane = threadIdx.x & 63;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < a.n; i += (int64_t)gridDim.x * 4) {
    const uint32_t r = row_of(a, i);
    const bool there = r < a.v;
    const T* w = static_cast<const T*>(a.weight) + (there ? (int64_t)r * a.h : 0);
    T* out = static_cast<T*>(a.out) + i * a.h;
    for (int c0 = lane * VEC; c0 < a.h; c0 += kPieces * 64 * VEC) {
      V x[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; k++) x[k] = *reinterpret_cast<const V*>(w + min(c0 + k * 64 * VEC, a.h - VEC));
#pragma unroll
      for (int k = 0; k < kPieces; k++) {
#pragma unroll
        for (int j = 0; j < VEC; j++) x[k][j] = there ? (T)((float)x[k][j] * a.scale) : (T)0.0f;
      }
#pragma unroll
      for (int k = 0; k < kPieces; k++)
        if (c0 + k * 64 * VEC < a.h) *reinterpret_cast<V*>(out + c0 + k * 64 * VEC) = x[k];
    }
  }
}

// ---------------------------------------------------------------------------
// Zeros for the rows that do not occur.  They are most of the gradient's bytes, and need
// nothing of the sort: they are written by further workgroups of the sort's own launches,
// a share by each, while its few workgroups wait on memory and on each other.  (Rows that
// occur are written twice, at most as many as there are tokens.)
// ---------------------------------------------------------------------------
struct ZeroArgs {
  char* to;                // NULL: nothing to write
  int64_t from, until;     // this launch's bytes, in whole pieces of kZeroPiece but for the end
  int first;               // the launch's first workgroup that writes
};
constexpr int64_t kZeroPiece = 64 * 1024;

template <int THREADS> __device__ __forceinline__ void write_zeros(const ZeroArgs& z, int block) {
  for (int64_t at = z.from + block * kZeroPiece; at < z.until; at += ((int64_t)gridDim.x - z.first) * kZeroPiece) {
    char* to = z.to + at + threadIdx.x * 16;
    const i32x4 zeros = {0, 0, 0, 0};
    if (at + kZeroPiece <= z.until) {
#pragma unroll
      for (int k = 0; k < (int)kZeroPiece / (16 * THREADS); k++) *reinterpret_cast<i32x4*>(to + k * 16 * THREADS) = zeros;
      continue;
    }
    const int64_t whole = z.until / 16 * 16;   // the last piece, and the bytes after its last whole 16
    for (int64_t i = at + threadIdx.x * 16; i < whole; i += 16 * THREADS) *reinterpret_cast<i32x4*>(z.to + i) = zeros;
    if (threadIdx.x < z.until - whole) z.to[whole + threadIdx.x] = 0;
  }
}
// A gradient that is not 16-byte aligned.
__global__ __launch_bounds__(256) void embed_zero_kernel(uint16_t* gw, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) gw[i] = 0;
}

// ---------------------------------------------------------------------------
// Stable radix sort of (id, token), kSortBits a pass.
// ---------------------------------------------------------------------------
struct SortArgs {
  EmbedArgs e;
  ZeroArgs z;
  int shift, first;            // bits already sorted; first pass: keys come from the ids
  int passes, parts;           // sort_parts_kernel
  const uint32_t* keys;
  const uint32_t* at;
  uint32_t* keys_out;
  uint32_t* at_out;
  uint32_t* hist;              // [kSortBins][blocks]
  int blocks;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int64_t i) {
  return a.first ? row_of(a.e, i) : a.keys[i];
}

// Ranks items by digit within their wave, a round of 64 after the other: the lanes of a round with the same digit find
// each other by ballots, and the first of them counts for all.  bins: the wave's counts, zeroed before, its items by
// digit after.
__device__ __forceinline__ uint32_t round_rank(uint32_t key, bool here, int shift, uint32_t* bins, int lane) {
  const uint32_t digit = (key >> shift) & (kSortBins - 1);
  uint64_t same = __ballot(here);
#pragma unroll
  for (int b = 0; b < kSortBits; b++) {
    const bool bit = (digit >> b) & 1;
    const uint64_t m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  const uint64_t below = same & ((uint64_t(1) << lane) - 1);
  const uint32_t rank = here ? bins[digit] + (uint32_t)__popcll(below) : 0u;
  wave_lds_sync();
  if (here && below == 0) bins[digit] += (uint32_t)__popcll(same);
  wave_lds_sync();
  return rank;
}

// Up to kSortAlone tokens, one launch.  Equal ids have to be neighbours, no more: ids fall into parts by a hash, a
// workgroup reads all ids, keeps its part's (in their order), sorts those in LDS, and writes them after the parts
// before its own, whose ids it has counted too.  So no workgroup waits for another, and with Zipf's ids the one that
// holds the most frequent sorts an eighth of the tokens.  (16000 tokens, V = 32000: one workgroup for all 43 us; three
// launches a pass 66 us for 32768.)  Tokens without a row come last.
__global__ __launch_bounds__(1024) void sort_parts_kernel(SortArgs a) {
  constexpr int kRounds = kSortAlone / 1024;
  __shared__ uint32_t keys[kSortAlone];
  __shared__ uint16_t ats[kSortAlone];
  __shared__ uint32_t bins[16][kSortBins];
  __shared__ uint32_t totals[16], before[16], none[16];
  if ((int)blockIdx.x >= a.z.first) {
    write_zeros<1024>(a.z, (int)blockIdx.x - a.z.first);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = (int)a.e.n;
  const uint32_t v = (uint32_t)a.e.v, own = blockIdx.x;
  const uint64_t lanes_below = (uint64_t(1) << lane) - 1;
  uint32_t key[kRounds], at[kRounds], rank[kRounds];
  {
    // a wave's ids are neighbours
    const int rounds = (n + 1023) / 1024, i0 = wave * rounds * 64, n_here = min(max(n - i0, 0), rounds * 64);
    uint32_t mine = 0, less = 0, missing = 0;
#pragma unroll
    for (int k = 0; k < kRounds; k++) key[k] = k * 64 + lane < n_here ? row_of(a.e, i0 + k * 64 + lane) : v;
#pragma unroll
    for (int k = 0; k < kRounds; k++) {
      if (k >= rounds) break;
      const bool here = k * 64 + lane < n_here;
      const uint32_t part = ((key[k] * 2654435761u) >> 16) % (uint32_t)a.parts;
      const uint64_t m = __ballot(here && key[k] < v && part == own);
      rank[k] = (m >> lane) & 1 ? mine + (uint32_t)__popcll(m & lanes_below) : 0xFFFFFFFFu;
      mine += (uint32_t)__popcll(m);
      less += (uint32_t)__popcll(__ballot(here && key[k] < v && part < own));
      missing += (uint32_t)__popcll(__ballot(here && key[k] == v));
    }
    if (lane == 0) {
      totals[wave] = mine;
      before[wave] = less;
      none[wave] = missing;
    }
    __syncthreads();
    uint32_t base = 0;
    for (int w = 0; w < wave; w++) base += totals[w];
#pragma unroll
    for (int k = 0; k < kRounds; k++) {
      if (k >= rounds) break;
      if (rank[k] == 0xFFFFFFFFu) continue;
      keys[base + rank[k]] = key[k];
      ats[base + rank[k]] = (uint16_t)(i0 + k * 64 + lane);
    }
  }
  uint32_t count = 0, start = 0, missing = 0;
  for (int w = 0; w < 16; w++) {
    count += totals[w];
    start += before[w];
    missing += none[w];
  }
  if (own == 0)   // the tokens without a row, after all others
    for (uint32_t i = tid; i < missing; i += 1024) {
      a.keys_out[n - missing + i] = v;
      a.at_out[n - missing + i] = 0;
    }
  __syncthreads();
  const int rounds = ((int)count + 1023) / 1024, i0 = wave * rounds * 64, n_here = min(max((int)count - i0, 0), rounds * 64);
#pragma unroll
  for (int k = 0; k < kRounds; k++) {
    if (k * 64 + lane >= n_here) continue;
    key[k] = keys[i0 + k * 64 + lane];
    at[k] = ats[i0 + k * 64 + lane];
  }
  for (int pass = 0; pass < a.passes; pass++) {
    const int shift = pass * kSortBits;
    for (int k = tid; k < 16 * kSortBins; k += 1024) bins[k / kSortBins][k % kSortBins] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; k++) {
      if (k >= rounds) break;
      rank[k] = round_rank(key[k], k * 64 + lane < n_here, shift, bins[wave], lane);
    }
    __syncthreads();
    // exclusive scan in the order (digit, wave): a thread's digit over the waves, then the digits
    uint32_t sum = 0, x = 0;
    if (tid < kSortBins) {
#pragma unroll
      for (int w = 0; w < 16; w++) {
        const uint32_t c = bins[w][tid];
        bins[w][tid] = sum;
        sum += c;
      }
      x = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = __shfl_up(x, o);
        if (lane >= o) x += y;
      }
      if (lane == 63) totals[wave] = x;
    }
    __syncthreads();
    if (tid < kSortBins) {
      uint32_t base = x - sum;
      for (int w = 0; w < wave; w++) base += totals[w];
#pragma unroll
      for (int w = 0; w < 16; w++) bins[w][tid] += base;
    }
    __syncthreads();
    const bool last = pass == a.passes - 1;
#pragma unroll
    for (int k = 0; k < kRounds; k++) {
      if (k * 64 + lane >= n_here) continue;
      const uint32_t to = bins[wave][(key[k] >> shift) & (kSortBins - 1)] + rank[k];
      if (last) {
        a.keys_out[start + to] = key[k];
        a.at_out[start + to] = at[k];
      } else {
        keys[to] = key[k];
        ats[to] = (uint16_t)at[k];
      }
    }
    if (last) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; k++) {
      if (k * 64 + lane >= n_here) continue;
      key[k] = keys[i0 + k * 64 + lane];
      at[k] = ats[i0 + k * 64 + lane];
    }
    __syncthreads();
  }
}
static_assert(kSortBins == 8 * 64, "the scan's digits are eight waves'");

// More tokens, three launches a pass: counts by workgroup, an exclusive scan of them in
// the order (digit, workgroup), then every item to its place.  A workgroup of W waves
// takes 512 W items.
constexpr int kWaveRounds = 8;
template <int W> __global__ __launch_bounds__(64 * W) void sort_count_kernel(SortArgs a) {
  __shared__ uint32_t bins[kSortBins];
  if ((int)blockIdx.x >= a.z.first) {
    write_zeros<64 * W>(a.z, (int)blockIdx.x - a.z.first);
    return;
  }
  const int tid = threadIdx.x;
  for (int k = tid; k < kSortBins; k += 64 * W) bins[k] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * (64 * W * kWaveRounds);
#pragma unroll
  for (int k = 0; k < kWaveRounds; k++) {
    const int64_t i = i0 + k * 64 * W + tid;
    if (i < a.e.n) atomicAdd(&bins[(sort_key(a, i) >> a.shift) & (kSortBins - 1)], 1u);   // counts: any order
  }
  __syncthreads();
  for (int k = tid; k < kSortBins; k += 64 * W) a.hist[(int64_t)k * a.blocks + blockIdx.x] = bins[k];
}

// In place, one workgroup.
__global__ __launch_bounds__(1024) void sort_scan_kernel(SortArgs a) {
  __shared__ uint32_t waves[16];
  if ((int)blockIdx.x >= a.z.first) {
    write_zeros<1024>(a.z, (int)blockIdx.x - a.z.first);
    return;
  }
  const int64_t n4 = (int64_t)kSortBins / 4 * a.blocks;   // four counts a thread
  const int tid = threadIdx.x, lane = tid & 63;
  i32x4* hist = reinterpret_cast<i32x4*>(a.hist);
  uint32_t before = 0;
  i32x4 ahead = tid < n4 ? hist[tid] : i32x4{0, 0, 0, 0};
  for (int64_t i0 = 0; i0 < n4; i0 += 1024) {
    const i32x4 own = ahead;
    if (i0 + 1024 < n4) ahead = i0 + 1024 + tid < n4 ? hist[i0 + 1024 + tid] : i32x4{0, 0, 0, 0};
    const uint32_t sum = (uint32_t)(own[0] + own[1] + own[2] + own[3]);
    uint32_t x = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    if (lane == 63) waves[tid >> 6] = x;
    __syncthreads();
    uint32_t base = before, total = 0;
#pragma unroll
    for (int w = 0; w < 16; w++) {
      if (w < tid >> 6) base += waves[w];
      total += waves[w];
    }
    i32x4 out;
    out[0] = (int)(base + x - sum);
#pragma unroll
    for (int j = 1; j < 4; j++) out[j] = out[j - 1] + own[j - 1];
    if (i0 + tid < n4) hist[i0 + tid] = out;
    before += total;
    __syncthreads();
  }
}

template <int W> __global__ __launch_bounds__(64 * W) void sort_place_kernel(SortArgs a) {
  __shared__ uint32_t bins[W][kSortBins];
  if ((int)blockIdx.x >= a.z.first) {
    write_zeros<64 * W>(a.z, (int)blockIdx.x - a.z.first);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int k = tid; k < W * kSortBins; k += 64 * W) bins[k / kSortBins][k % kSortBins] = 0;
  const int64_t i0 = (int64_t)(blockIdx.x * W + wave) * (64 * kWaveRounds);
  const int n_here = (int)min(max(a.e.n - i0, (int64_t)0), (int64_t)64 * kWaveRounds);
  uint32_t key[kWaveRounds], at[kWaveRounds], rank[kWaveRounds];
#pragma unroll
  for (int k = 0; k < kWaveRounds; k++) {
    const int64_t i = i0 + k * 64 + lane;
    const bool here = k * 64 + lane < n_here;
    key[k] = here ? sort_key(a, i) : 0u;
    at[k] = here && !a.first ? a.at[i] : (uint32_t)i;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWaveRounds; k++) rank[k] = round_rank(key[k], k * 64 + lane < n_here, a.shift, bins[wave], lane);
  __syncthreads();
  for (int d = tid; d < kSortBins; d += 64 * W) {
    uint32_t s = a.hist[(int64_t)d * a.blocks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < W; w++) {
      const uint32_t c = bins[w][d];
      bins[w][d] = s;
      s += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWaveRounds; k++) {
    if (k * 64 + lane >= n_here) continue;
    const uint32_t to = bins[wave][(key[k] >> a.shift) & (kSortBins - 1)] + rank[k];
    a.keys_out[to] = key[k];
    a.at_out[to] = at[k];
  }
}

// ---------------------------------------------------------------------------
// Sums of runs, by chunks of 16 tokens (32 beyond 16384, more where there would be over 4096
// chunks).  N = 8192 above in chunks of 8 / 16 / 32 / 64: runs 36 / 36 / 36 / 79 us, joins 15 /
// 9 / 7 / 6; N = 1000, H = 4096: runs 7 / 9 / 14 / 57.
// ---------------------------------------------------------------------------
struct RunArgs {
  const uint32_t* keys;        // equal ones next to each other; tokens without a row last
  const uint32_t* at;
  int64_t n, v;
  int h, chunk;
  int64_t n_chunks;
  float scale;
  int accumulate;
  const void* grad;
  void* gw;
  float* part;                 // [2][n_chunks][h]: what a chunk's first run adds to one begun before it, and its
                               // last run's sum where that goes on
};

template <typename O, int VEC>
__device__ __forceinline__ void put_row(const RunArgs& a, uint32_t row, int c, const float (&s)[VEC]) {
  typedef O V __attribute__((ext_vector_type(VEC)));
  V* to = reinterpret_cast<V*>(static_cast<O*>(a.gw) + (int64_t)row * a.h + c);
  V o;
  if (a.accumulate) {
    o = *to;
#pragma unroll
    for (int j = 0; j < VEC; j++) o[j] = (O)fmaf(s[j], a.scale, (float)o[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j++) o[j] = (O)(s[j] * a.scale);
  }
  *to = o;
}

// VEC elements as they are loaded, in a register type: 16 bytes, or one element as its value.
template <typename T, int VEC> struct Loaded {
  i32x4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const i32x4*>(p); }
  __device__ __forceinline__ float get(int j) const {
    typedef T V __attribute__((ext_vector_type(VEC)));
    return (float)__builtin_bit_cast(V, raw)[j];
  }
};
template <typename T> struct Loaded<T, 1> {
  float raw;
  __device__ __forceinline__ void load(const T* p) { raw = (float)*p; }
  __device__ __forceinline__ float get(int) const { return raw; }
};

// One chunk of sorted tokens by 256 VEC columns; the rows of kAhead tokens are in flight at a time.
constexpr int kAhead = 8;   // divides 64
template <typename T, typename O, int VEC> __global__ __launch_bounds__(256) void embed_runs_kernel(RunArgs a) {
  const int64_t chunk = blockIdx.x, i0 = chunk * a.chunk, i1 = min(i0 + a.chunk, a.n);
  const int lane = threadIdx.x & 63, c = ((int)blockIdx.y * 256 + (int)threadIdx.x) * VEC;
  uint32_t key = a.keys[i0];
  // whole waves only: a lane past the row's end holds tokens for the others (and reads the row's last piece)
  if (c - lane * VEC >= a.h || key >= a.v) return;
  const bool in = c < a.h;
  const int c_read = min(c, a.h - VEC);
  float s[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) s[j] = 0.0f;
  bool inner = i0 == 0 || a.keys[i0 - 1] != key;   // the run began here
  for (int64_t i = i0; i < i1; i += 64) {
    // a lane's token and the key after its own, for the wave's scalar registers
    const int64_t mine = min(i + lane, i1 - 1);   // past the chunk's end its last token again, not added
    const int at = (int)a.at[mine], after = (int)(mine + 1 < a.n ? a.keys[mine + 1] : (uint32_t)a.v);
    const int here = (int)min(i1 - i, (int64_t)64);
    for (int b = 0; b < here; b += kAhead) {
      Loaded<T, VEC> g[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; k++)
        g[k].load(static_cast<const T*>(a.grad) + (int64_t)(uint32_t)__builtin_amdgcn_readlane(at, b + k) * a.h + c_read);
      // (else the compiler moves each load down to its use, and they wait for memory one after the other)
#pragma unroll
      for (int k = 0; k < kAhead; k++) asm volatile("" : "+v"(g[k].raw));
#pragma unroll
      for (int k = 0; k < kAhead; k++) {
        if (b + k >= here || key >= a.v) return;
#pragma unroll
        for (int j = 0; j < VEC; j++) s[j] += g[k].get(j);
        const uint32_t next = (uint32_t)__builtin_amdgcn_readlane(after, b + k);
        if (next == key && i + b + k + 1 < i1) continue;
        if (inner && next != key) {
          if (in) put_row<O, VEC>(a, key, c, s);
        } else if (in) {
          float* p = a.part + ((inner ? a.n_chunks : 0) + chunk) * a.h + c;
#pragma unroll
          for (int j = 0; j < VEC; j++) p[j] = s[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; j++) s[j] = 0.0f;
        key = next;
        inner = true;
      }
    }
  }
}

// Runs that begin in a chunk and end in another, by 64 VEC columns: the parts in four ranges, a wave each.
template <typename O, int VEC> __global__ __launch_bounds__(256) void embed_join_kernel(RunArgs a) {
  typedef float V __attribute__((ext_vector_type(VEC)));
  __shared__ V sums[4][64];
  const int64_t chunk = blockIdx.x, i0 = chunk * a.chunk, i1 = i0 + a.chunk;
  if (i1 >= a.n) return;
  const uint32_t key = a.keys[i1 - 1];
  if (key >= a.v || a.keys[i1] != key) return;
  if (i0 > 0 && a.keys[i0] == key && a.keys[i0 - 1] == key) return;   // begun before
  // the chunks after it that begin with the same key: a lane looks at each
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t last = chunk + 1;
  for (;;) {
    const int64_t k = last + 1 + lane;
    const uint64_t goes_on = __ballot(k < a.n_chunks && a.keys[min(k * a.chunk, a.n - 1)] == key);
    const int more = goes_on == ~uint64_t(0) ? 64 : __ffsll((unsigned long long)~goes_on) - 1;
    last += more;
    if (more < 64) break;
  }
  const int c = ((int)blockIdx.y * 64 + lane) * VEC, at = min(c, a.h - VEC);
  // part 0 is this chunk's own, the others' follow
  const int64_t parts = last - chunk + 1, p0 = parts * wave / 4, p1 = parts * (wave + 1) / 4;
  V s;
#pragma unroll
  for (int j = 0; j < VEC; j++) s[j] = 0.0f;
  for (int64_t p = p0; p < p1; p += 8) {
    V v[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {   // eight in flight; past the last one it again, not added
      const int64_t q = min(p + k, p1 - 1);
      v[k] = *reinterpret_cast<const V*>(a.part + ((q == 0 ? a.n_chunks : q) + chunk) * a.h + at);
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (p + k < p1) s += v[k];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= a.h) return;
  const V all = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
  float out[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) out[j] = all[j];
  put_row<O, VEC>(a, key, c, out);
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

void plan_embedding_backward(EmbedPlan* p) {
  int bits = 1;
  while ((p->v >> bits) != 0) bits++;      // of the key v
  p->passes = (bits + kSortBits - 1) / kSortBits;
  p->sort_parts = p->sort_blocks = 0;
  if (p->n <= kSortAlone) {
    const int64_t parts = (p->n + 511) / 512;
    p->sort_parts = (int)(parts < 32 ? parts : 32);
  } else {
    // small workgroups: 32768 tokens' last launch of a pass took 17 us by workgroups of 16 waves.  The scan, one
    // workgroup's, has a count for each digit and workgroup.
    p->sort_waves = p->n <= (1 << 18) ? 4 : 16;
    const int64_t items = 64 * kWaveRounds * p->sort_waves;
    p->sort_blocks = (int)((p->n + items - 1) / items);
  }
  p->chunk = p->n <= 16384 ? 16 : 32;
  while (p->chunk < (1 << 20) && p->n / p->chunk > 4096) p->chunk *= 2;
  p->n_chunks = (p->n + p->chunk - 1) / p->chunk;
  size_t o = 0;
  for (int k = 0; k < (p->sort_blocks > 0 ? 2 : 1); k++) {
    p->w_keys[k] = o;
    o += up256(size_t(p->n) * 4);
    p->w_at[k] = o;
    o += up256(size_t(p->n) * 4);
  }
  p->w_hist = o;
  o += up256(size_t(kSortBins) * p->sort_blocks * 4);
  p->w_part = o;
  o += up256(size_t(2) * p->n_chunks * p->h * 4);
  p->w_bytes = o > 0 ? o : 256;
}

static size_t bytes_of(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }
static bool whole16(const void* p, int64_t h, int dtype) {   // rows of whole, aligned 16-byte pieces
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (h * bytes_of(dtype)) % 16 == 0;
}

static EmbedArgs embed_args(const EmbedPlan& p, const void* ids) {
  EmbedArgs a{};
  a.ids = ids;
  a.ids_i32 = p.ids_i32 ? 1 : 0;
  a.n = p.n;
  a.v = p.v;
  a.ignore_index = p.ignore_index;
  a.h = p.h;
  a.scale = p.scale;
  return a;
}

template <typename T> static void embed_forward_t(const EmbedPlan& p, const EmbedArgs& a, hipStream_t st) {
  const int64_t need = (p.n + 3) / 4;
  const unsigned wgs = (unsigned)(need < 65536 ? need : 65536);
  if (whole16(a.weight, p.h, p.dtype) && whole16(a.out, p.h, p.dtype))
    embed_fwd_kernel<T, 16 / sizeof(T)><<<wgs, 256, 0, st>>>(a);
  else
    embed_fwd_kernel<T, 1><<<wgs, 256, 0, st>>>(a);
}

hipError_t launch_embedding_forward(const EmbedPlan& p, const void* ids, const void* weight, void* out, hipStream_t st) {
  if (p.n == 0) return hipSuccess;
  EmbedArgs a = embed_args(p, ids);
  a.weight = weight;
  a.out = out;
  if (p.dtype == FLCE_BF16) embed_forward_t<bf16>(p, a, st);
  else if (p.dtype == FLCE_F16) embed_forward_t<f16>(p, a, st);
  else embed_forward_t<float>(p, a, st);
  return hipGetLastError();
}

template <typename T, typename O> static void embed_runs_t(const EmbedPlan& p, const RunArgs& a, hipStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const bool vec = whole16(a.grad, p.h, p.dtype) && p.h % kVec == 0 &&
                   (reinterpret_cast<uintptr_t>(a.gw) & (kVec * sizeof(O) - 1)) == 0;
  const int per = 256 * (vec ? kVec : 1);
  const dim3 grid((unsigned)p.n_chunks, (unsigned)((p.h + per - 1) / per));
  if (vec) embed_runs_kernel<T, O, kVec><<<grid, 256, 0, st>>>(a);
  else embed_runs_kernel<T, O, 1><<<grid, 256, 0, st>>>(a);
  if (p.h % 4 == 0 && (reinterpret_cast<uintptr_t>(a.gw) & (4 * sizeof(O) - 1)) == 0)
    embed_join_kernel<O, 4><<<dim3((unsigned)p.n_chunks, (unsigned)((p.h + 255) / 256)), 256, 0, st>>>(a);
  else
    embed_join_kernel<O, 1><<<dim3((unsigned)p.n_chunks, (unsigned)((p.h + 63) / 64)), 256, 0, st>>>(a);
}

template <typename T> static void embed_runs_o(const EmbedPlan& p, const RunArgs& a, hipStream_t st) {
  if (p.grad_dtype == FLCE_BF16) embed_runs_t<T, bf16>(p, a, st);
  else if (p.grad_dtype == FLCE_F16) embed_runs_t<T, f16>(p, a, st);
  else embed_runs_t<T, float>(p, a, st);
}

hipError_t launch_embedding_backward(const EmbedPlan& p, const void* ids, const void* grad, void* grad_weight, char* ws,
                                     hipStream_t st) {
  SortArgs s{};
  s.e = embed_args(p, ids);
  const int64_t bytes = p.v * p.h * (int64_t)bytes_of(p.grad_dtype);
  const bool zeros = !p.accumulate && (reinterpret_cast<uintptr_t>(grad_weight) & 15) == 0;
  if (!p.accumulate && !zeros)
    embed_zero_kernel<<<4096, 256, 0, st>>>(static_cast<uint16_t*>(grad_weight), bytes / 2);
  // the launches' shares of the zeros
  const bool alone = p.sort_blocks == 0;
  const int launches = alone ? 1 : 3 * p.passes;
  const int64_t pieces = zeros ? (bytes + kZeroPiece - 1) / kZeroPiece : 0;
  int done = 0;
  auto blocks_with_zeros = [&](int sorting) {
    const int64_t from = pieces * done / launches, until = pieces * (done + 1) / launches;
    done++;
    s.z.to = static_cast<char*>(grad_weight);
    s.z.from = from * kZeroPiece;
    s.z.until = until * kZeroPiece < bytes ? until * kZeroPiece : bytes;
    s.z.first = sorting;
    const int64_t n = until - from;
    return (unsigned)(sorting + (n < 65536 ? n : 65536));
  };
  s.passes = p.passes;
  s.parts = p.sort_parts;
  if (alone) {
    s.first = 1;
    s.keys_out = reinterpret_cast<uint32_t*>(ws + p.w_keys[0]);
    s.at_out = reinterpret_cast<uint32_t*>(ws + p.w_at[0]);
    const unsigned blocks = blocks_with_zeros(p.sort_parts);
    if (blocks > 0) sort_parts_kernel<<<blocks, 1024, 0, st>>>(s);
  } else {
    s.hist = reinterpret_cast<uint32_t*>(ws + p.w_hist);
    s.blocks = p.sort_blocks;
    int to = 0;
    for (int k = 0; k < p.passes; k++, to ^= 1) {
      s.shift = k * kSortBits;
      s.first = k == 0;
      s.keys = reinterpret_cast<const uint32_t*>(ws + p.w_keys[to ^ 1]);
      s.at = reinterpret_cast<const uint32_t*>(ws + p.w_at[to ^ 1]);
      s.keys_out = reinterpret_cast<uint32_t*>(ws + p.w_keys[to]);
      s.at_out = reinterpret_cast<uint32_t*>(ws + p.w_at[to]);
      unsigned blocks = blocks_with_zeros(p.sort_blocks);
      if (p.sort_waves == 4) sort_count_kernel<4><<<blocks, 256, 0, st>>>(s);
      else sort_count_kernel<16><<<blocks, 1024, 0, st>>>(s);
      blocks = blocks_with_zeros(1);
      sort_scan_kernel<<<blocks, 1024, 0, st>>>(s);
      blocks = blocks_with_zeros(p.sort_blocks);
      if (p.sort_waves == 4) sort_place_kernel<4><<<blocks, 256, 0, st>>>(s);
      else sort_place_kernel<16><<<blocks, 1024, 0, st>>>(s);
    }
  }
  if (p.n == 0) return hipGetLastError();
  RunArgs a{};
  a.keys = s.keys_out;
  a.at = s.at_out;
  a.n = p.n;
  a.v = p.v;
  a.h = p.h;
  a.chunk = p.chunk;
  a.n_chunks = p.n_chunks;
  a.scale = p.scale;
  a.accumulate = p.accumulate ? 1 : 0;
  a.grad = grad;
  a.gw = grad_weight;
  a.part = reinterpret_cast<float*>(ws + p.w_part);
  if (p.dtype == FLCE_BF16) embed_runs_o<bf16>(p, a, st);
  else if (p.dtype == FLCE_F16) embed_runs_o<f16>(p, a, st);
  else embed_runs_o<float>(p, a, st);
  return hipGetLastError();
}

}  // namespace flce
