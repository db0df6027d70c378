// window_attn.cu -- causal attention of packed prompts, with an optional
// sliding window and a few first tokens that stay visible.
//
// Row i of a sequence of nq rows and nk keys stands at position
// p = nk - nq + i and sees key j iff j <= p and (no window, or j > p - window,
// or j < sinks):   O = softmax_j(scale <Q, K_j>) V, zeros where nothing is seen.
//
// What bounds it: 4 * D * Hq products per visible (row, key) pair, so the
// tensor cores; beside them one exponential per pair and query head.  Hence:
//  * A tile is 128 query rows of one KV head: 128/G positions times the G query
//    heads that share it, so short prompts and window edges waste few rows
//    and the K/V stream of a tile serves all G heads.
//  * Both products run as tcgen05.mma with fp32 accumulators in tensor memory:
//    S = Q K^T from shared memory, O += P V with P (bf16) written over S in
//    tensor memory by the softmax threads, one row a thread.
//  * D = 128: a CTA carries two tiles (256 rows) with a softmax warpgroup each;
//    the tensor cores work on one tile's products while the other's softmax
//    runs, and each K/V block of 128 keys is fetched once for both.
//    D = 256: O alone takes half of tensor memory, so a CTA carries one tile
//    with two S buffers: S of the next block is computed during the softmax of
//    this one, whose rows two threads share (half of the keys each; they
//    exchange one maximum a block).  Blocks are 128 keys there too: with 64, S
//    takes twice the instructions, each as long to issue (about 55 clocks) as
//    to execute.
//  * Only blocks that some row of the CTA's tiles sees are visited; behind a
//    window they begin at the first key seen, and up to 32 always visible first
//    keys take the place of keys before it in the first block, so that they cost
//    no block (8192 rows of 32 heads, window 1024, 4 first keys: 129 -> 122 us).
//    (Blocks cut to whole groups of 32 keys cost every other block more than
//    they save: 138 us.)
//  * One warp streams K with TMA, one V, each into a ring of its own; another
//    fetches the next tiles' queries as soon as the last S product is done, and
//    tells the issuing warp the item's size: what that warp does between two
//    products is on every tile's path (its own look-up: 373 us against 354 for
//    8192 rows of 32 heads, causal).
//  * Keys past a sequence's end belong to others.  Scores against them are
//    masked; their values are not fetched (pieces of 32 keys, the last filled up
//    with zeros by the issuing warp, older values behind it), as zeroing up to a
//    whole block there cost the longest item 1 us.
//  * The maximum that P refers to is raised only when a block exceeds it by
//    more than 2^8, so O is rarely rescaled; P is rounded to bf16 (relative
//    2^-8 at most, as the second product's operand), sums are fp32.
// Measured, on the GPU: 8000 rows of 24/4 heads of 256, causal: 465-495 us over
// several GPUs, 1.59-1.69 PFLOP/s (bound by the tensor cores and by power; 515-524
// us as single calls, 1.50-1.53); 8192 rows of 32/8 heads of 128, causal: 355 us, 1.55
// PFLOP/s (379 as a call), with a window of 1024 and 4 first keys 117 us (121; the
// softmax of two tiles, about 1750 clocks a block each, and its hand-overs); 2048
// rows behind 6144 keys, 32/8 heads of 128: 207 us as a call, 1.16 PFLOP/s (1.7
// items a CTA); seven prompts of 2 to 901 rows, 32/8 heads of 128: 19.5 us (three
// items of 1 to 8 blocks a CTA; start 2600 clocks, end of an item 3200, a block 1850).
#include "paged.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace attn {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // attn.cu
}
namespace window {

constexpr int ROWS = 128;           // rows of a tile (TMEM lanes)
constexpr int BN = 128;             // keys of a block
constexpr int PIECE = 32;           // keys of a smaller copy; first keys that may share a block with others
constexpr int MAX_B = 4096;
constexpr float RESCALE = 8.f;      // log2 of the largest P against an old maximum
// Shared memory: barriers, scan totals (320), the CTA's items (384), the item
// (448), halves' exchange (512), prefix sums (2560; after the ring if longer), then the query
// tiles and the ring.
constexpr int HEADER = 3072, PREFIX = 2560, SCAN = 320, ORDER = 384, INFO = 448;
// Up to this many sequences and rounds, the items go longest first.
constexpr int MAX_SORTED = 32, MAX_SORTED_ROUNDS = 12;
constexpr int SORT_UNIT = 64;       // keys that count as equally long

// Two tiles a CTA (D = 128), or one with two S buffers and two threads a row.
template <int D, int TILES>
struct Cfg {
  static constexpr int NT = TILES;
  static constexpr int NSB = TILES == 2 ? 1 : 2;  // S buffers per tile
  static constexpr int SOFT = 8;                  // softmax warps
  static constexpr int HALVES = TILES == 2 ? 1 : 2;  // threads that share a row
  // Ring slots: a whole K or V block at D = 128, at D = 256 half of its columns
  // (K) or of its keys (V).  (Quarters are freed earlier, but the issuing warp's
  // waits for them cost more: 526 against 473 us for 8000 rows of 24 heads.)
  static constexpr int SLOT = 32768;
  static constexpr int PARTS = BN * D * 2 / SLOT;  // slots of a K block (of a V block)
  static constexpr int KG = D / 64 / PARTS;        // 64-column groups of a K slot
  static constexpr int VK = BN / PARTS;            // keys of a V slot
  static constexpr int THREADS = (SOFT + 4) * 32;
  static constexpr int QBYTES = ROWS * D * 2;
  static constexpr int RING = HEADER + NT * QBYTES;
  // slots of the K and the V ring: 160 KB, or 128 beside long prefix sums
  static constexpr int NK = 2, NV = 3, LESS = 2;
  static_assert((NK + NV) * SLOT == 160 * 1024 && 2 * LESS * SLOT == 128 * 1024, "ring");
  // tensor memory: O per tile, then the S buffers (P over S)
  static constexpr uint32_t TO = 0, TS = NT * D;
  static_assert(NT * D + NT * NSB * BN <= 512, "tensor memory");
};

struct Params {
  sv_rows o;
  const int *cu_q, *cu_k;
  unsigned *err;
  int B, Tq, Tk, Hkv, G, PT;  // PT: positions per tile
  uint32_t by_span;  // 2^32 over the positions of an item
  int most;          // items a KV head that sequences without common rows can have
  float sl2e;
  int window, sinks;
  int few_slots;  // long prefix sums take the place of some
  int stall;      // test aid: the first slot of the K ring never fills
};

struct Item {
  int h, q0, k0;     // KV head; first row of the packed queries and keys
  int rows;          // positions of the item
  int p0, nk;        // position of its first row; keys of the sequence
  // Blocks: ns over the first keys, then those from key w0 on; n in all.  Up to
  // PIECE first keys far from the window (ns = 0, w0 > 0, sinks) need no block:
  // keys 0..PIECE-1 stand in the first block's first rows, for w0..w0+PIECE-1.
  int ns, skip, n;
  __device__ __forceinline__ int base(int j) const { return j * BN + (j < ns ? 0 : skip); }
};

// Rows of sequence b (and its keys), 0 if its offsets are out of order or out of range.
__device__ __forceinline__ int rows_of(const Params &P, int b, int &nk) {
  const int q0 = P.cu_q[b], q1 = P.cu_q[b + 1], k0 = P.cu_k[b], k1 = P.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > P.Tq || k0 < 0 || k1 < k0 || k1 > P.Tk) {
    if (blockIdx.x == 0) atomicOr(P.err, ERR_INDEX);
    return 0;
  }
  nk = k1 - k0;
  return q1 - q0;
}

template <int NT>
__device__ __forceinline__ Item item_at(const Params &P, const int *pre, int id) {
  const int c = id / P.Hkv;
  int lo = 0, hi = P.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= c) lo = mid; else hi = mid - 1;
  }
  const int b = lo, span = P.PT * NT;
  Item it;
  it.h = id - c * P.Hkv;
  // a sequence's last tiles first: they see the most
  const int tile = pre[b + 1] - 1 - c;
  const int nq = P.cu_q[b + 1] - P.cu_q[b];
  it.k0 = P.cu_k[b];
  it.nk = P.cu_k[b + 1] - it.k0;
  const int row0 = tile * span;
  it.q0 = P.cu_q[b] + row0;
  it.rows = imin(span, nq - row0);
  it.p0 = it.nk - nq + row0;
  const int end = imax(0, it.p0 + it.rows);  // of the keys that some row sees
  const int start = P.window > 0 ? imin(end, imax(0, it.p0 - P.window + 1)) : 0;
  const int first = imin(P.sinks, end);
  it.ns = first > PIECE ? (first + BN - 1) / BN : 0;
  int w0 = first > PIECE || first == 0 ? start : imax(0, start - PIECE);
  if (w0 <= it.ns * BN) w0 = it.ns = 0;
  it.skip = w0 - it.ns * BN;
  it.n = it.ns + (end - w0 + BN - 1) / BN;
  return it;
}

// Place of this CTA's item of round k on the line of items (-1: none in this
// round).  Rounds alternate direction, so that the CTA with a round's longest
// item gets the next one's shortest; of sorted items the last round runs
// backwards: what it lacks is lacking to the first CTAs, who had the longest.
__device__ __forceinline__ int place_of(int k, int rounds, int items, bool sorted) {
  const int g = (int)gridDim.x;
  const int at = (k & 1) || (sorted && k + 1 == rounds) ? g - 1 - (int)blockIdx.x : (int)blockIdx.x;
  return k * g + at < items ? k * g + at : -1;
}

// The item at a place of the line that has all items by the position of their
// last row, in units of SORT_UNIT, the largest first; a warp's work, one lane a
// sequence (of nt items a KV head, whose first is at position `off`).
__device__ __forceinline__ void find_sorted(const Params &P, const int *pre, const int2 *where, int place, int *out) {
  const int lane = threadIdx.x & 31;
  const bool in = lane < P.B;
  const int nt = in ? pre[lane + 1] - pre[lane] : 0;
  const int off = in ? where[lane].x : 0, end = nt > 0 ? where[lane].y : 0;
  // items of this lane's sequence that end in unit v + 1 or later
  auto after = [&](int v) {
    const int e = (v + 1) * SORT_UNIT;
    // (the quotient may be off by one far out, but never falls as v rises)
    return end < e ? 0 : nt - imin((int)__umulhi((uint32_t)imax(0, e - off - 1), P.by_span), nt - 1);
  };
  const int q = place / P.Hkv, head = place - q * P.Hkv;
  // v: the unit that the item ends in, the smallest with no more than q after it
  int lo = 0, hi = __reduce_max_sync(0xffffffffu, end) / SORT_UNIT;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__reduce_add_sync(0xffffffffu, after(mid)) <= q) hi = mid; else lo = mid + 1;
  }
  const int later = after(lo), here = (lo > 0 ? after(lo - 1) : nt) - later;
  int x = here;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const int r = q - __reduce_add_sync(0xffffffffu, later) - (x - here);
  if (r >= 0 && r < here) *out = (pre[lane] + later + r) * P.Hkv + head;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void tma_load_4d(void *smem_dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

template <int D, int TILES>
__global__ void __launch_bounds__(Cfg<D, TILES>::THREADS, 1)
    window_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                  const __grid_constant__ CUtensorMap mapV,
                  const __grid_constant__ CUtensorMap mapKp, const __grid_constant__ CUtensorMap mapVp,
                  const Params P) {
  using C = Cfg<D, TILES>;
  constexpr int NT = C::NT, NSB = C::NSB, PARTS = C::PARTS, VK = C::VK, KG = C::KG, SLOT = C::SLOT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw;
  // The swizzled tiles need 1024-byte alignment, which the first dynamic byte
  // has in a kernel without static shared memory; five slots leave no room to
  // round up.
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, ERR_TIMEOUT);
    return;
  }
  uint64_t *full = reinterpret_cast<uint64_t *>(smem);  // [2][5] slots of the K ring, of the V ring
  uint64_t *empty = full + 10;     // [2][5]
  uint64_t *s_full = empty + 10;   // [2] per S buffer
  uint64_t *p_full = s_full + 2;   // [2] per S buffer: P written over it
  uint64_t *o_done = p_full + 2;   // [2] per S buffer: the second product of its P done
  uint64_t *o_free = o_done + 2;   // [NT] O read out
  uint64_t *q_full = o_free + 2;   // queries of the item landed
  uint64_t *q_free = q_full + 1;   // last S product of the item done
  uint64_t *idle = q_free + 1;
  uint64_t *p_half = idle + 1;     // [2] one S buffer: P of the first half of a block's keys written
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(p_half + 2);
  int *wsum = reinterpret_cast<int *>(smem + SCAN);
  int4 *info = reinterpret_cast<int4 *>(smem + INFO);  // of the item whose queries landed
  float *xchg = reinterpret_cast<float *>(smem + 512);  // [2][2 halves][ROWS] maxima, then sums
  int2 *where = reinterpret_cast<int2 *>(xchg);         // before: of up to 32 sequences, nk - nq and nk
  uint8_t *qs = smem + HEADER;
  uint8_t *ring = smem + C::RING;
  const int NK = P.few_slots ? C::LESS : C::NK, NV = P.few_slots ? C::LESS : C::NV;
  int *pre = reinterpret_cast<int *>(P.few_slots ? ring + 2 * C::LESS * SLOT : smem + PREFIX);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 10; ++i) {
      mbar_init(&full[i], 1 + (i == 0 ? P.stall : 0));
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4 * C::HALVES);
      mbar_init(&o_done[i], 1);
      mbar_init(&p_half[i], 4);
      mbar_init(&o_free[i], 4 * C::HALVES);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(idle, 1);
    fence_barrier_init();
  }
  if (warp == C::SOFT) {
    tc::tmem_alloc(tmem_slot, 512u);
    tc::tmem_relinquish();
  }
  // rows of the query tiles that no load writes stay zero
  const int used = P.PT * P.G;
  for (int x = tid; x < NT * (ROWS - used) * (D / 8); x += C::THREADS) {
    const int t = x / ((ROWS - used) * (D / 8)), y = x % ((ROWS - used) * (D / 8));
    const int r = used + y / (D / 8), c = y % (D / 8);
    *reinterpret_cast<uint4 *>(qs + t * C::QBYTES + (c >> 3) * ROWS * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  // Values of a block's rows past the sequence's end are not fetched: what
  // stands there meets probabilities of zero and has to be finite.
  for (int x = tid; x < NV * SLOT / 16; x += C::THREADS)
    reinterpret_cast<uint4 *>(ring + NK * SLOT)[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  pdl_wait();

  // ---- prefix sums of the sequences' items per KV head ----
  // Offsets that fall and rise again can name the same rows thousands of times:
  // the sums stay at the top instead of wrapping, and then no item is left.
  auto sum = [](int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); };
  int total = 0;
  for (int b0 = 0; b0 < P.B; b0 += C::THREADS) {
    const int b = b0 + tid;
    int nk = 0;
    const int nq = b < P.B ? rows_of(P, b, nk) : 0;
    const int nt = (nq + P.PT * NT - 1) / (P.PT * NT);
    int x = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = sum(x, y);
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < C::THREADS / 32; ++w) {
      if (w < warp) before = sum(before, wsum[w]);
      all = sum(all, wsum[w]);
    }
    if (b < P.B) pre[b] = sum(total, sum(before, x)) - nt;
    if (b < P.B && b < MAX_SORTED) where[b] = make_int2(nk - nq, nk);
    total = sum(total, all);
    __syncthreads();
  }
  if (total > P.most) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(P.err, ERR_INDEX);
    total = 0;
  }
  if (tid == 0) pre[P.B] = total;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const int items = total * P.Hkv;
  const int rounds = (items + (int)gridDim.x - 1) / (int)gridDim.x;
  // Longest first, if that pays: one sequence is in order already, many rounds
  // even out by themselves, and finding the order takes 2 us (seven prompts of
  // 2 to 901 rows: 2.9 items a CTA at D = 128, 22.1 -> 19.4 us; 2.1 at D = 256,
  // 22.7 -> 23.4; 16 prompts of 69 to 1500 rows, 2.9 pairs, 68 -> 57).  Whether
  // they are sorted stands behind the list: no role has a register to spare.
  int *order = reinterpret_cast<int *>(smem + ORDER);
  const bool sorted = P.B > 1 && P.B <= MAX_SORTED && 2 * items >= 5 * (int)gridDim.x && rounds <= MAX_SORTED_ROUNDS;
  if (tid == 0) order[MAX_SORTED_ROUNDS] = sorted;
  if (sorted) {
    static_assert(C::THREADS / 32 >= MAX_SORTED_ROUNDS, "a warp a round");
    if (warp < rounds) {
      const int place = place_of(warp, rounds, items, true);
      if (place >= 0)
        find_sorted(P, pre, where, place, order + warp);
      else if (lane == 0)
        order[warp] = -1;
    }
  }
  __syncthreads();
  auto item_id = [&](int k) { return order[MAX_SORTED_ROUNDS] ? order[k] : place_of(k, rounds, items, false); };

  if (warp >= C::SOFT) {
    // 384 threads start with 168 registers each: 128*72 + 256*216 is the same total
    setmaxnreg_dec<72>();
    if (warp == C::SOFT + 1 || warp == C::SOFT + 3) {
      // -------------------------------- K blocks, in the other V blocks --
      if (lane == 0) {
        const bool is_v = warp == C::SOFT + 3;
        uint64_t *landed = full + (is_v ? 5 : 0), *free = empty + (is_v ? 5 : 0);
        uint8_t *slots = ring + (is_v ? NK * SLOT : 0);
        const int NS = is_v ? NV : NK;
        bool ok = true;
        uint32_t q = 0, parity = 1;
        int slot = 0;
        for (int k = 0; k < rounds && ok; ++k) {
          const int id = item_id(k);
          if (id < 0) continue;
          const Item it = item_at<NT>(P, pre, id);
          for (int j = 0; j < it.n && ok; ++j) {
            const int key = it.k0 + it.base(j);
            const bool head = j == 0 && it.ns == 0 && it.skip > 0 && P.sinks > 0;
            // keys of the sequence in this block (keys past the end may land: they are masked)
            const int kept = is_v ? imin(BN, it.nk - it.base(j)) : BN;
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              if (ok) ok = mbar_wait(&free[slot], parity, P.err);
              if (!ok) break;
              uint8_t *at = slots + slot * SLOT;
              if (!head && kept == BN) {
                mbar_arrive_expect_tx(&landed[slot], SLOT);
                tma_load_4d(at, is_v ? &mapV : &mapK, 0, is_v ? key + x * VK : key, is_v ? 0 : x * KG, it.h, &landed[slot]);
              } else {  // PIECE keys and 64 columns at a time
                const int rows = is_v ? VK : BN, first = is_v ? x * VK : 0, group = is_v ? 0 : x * KG;
                const int groups = SLOT / (rows * 128), some = imin(rows, imax(0, kept - first) + PIECE - 1) / PIECE * PIECE;
                mbar_arrive_expect_tx(&landed[slot], (uint32_t)(groups * some * 128));
                for (int g = 0; g < groups; ++g)
                  for (int y = 0; y < some; y += PIECE)
                    tma_load_4d(at + (g * rows + y) * 128, is_v ? &mapVp : &mapKp, 0,
                                head && first + y == 0 ? it.k0 : key + first + y, group + g, it.h, &landed[slot]);
              }
              ++q;
              if (++slot == NS) {
                slot = 0;
                parity ^= 1;
              }
            }
          }
        }
        if (!ok) {  // no copy may outlive the CTA
          const uint32_t first = q > (uint32_t)NS ? q - NS : 0u;
          for (uint32_t qq = first; qq < q && mbar_wait(&landed[qq % NS], (qq / NS) & 1, P.err); ++qq) {
          }
        }
      }
      __syncwarp();
    } else if (warp == C::SOFT + 2) {
      // --------------------------------------------------- queries --
      if (lane == 0) {
        bool ok = true;
        uint32_t c = 0;  // items with work so far
        for (int k = 0; k < rounds && ok; ++k) {
          const int id = item_id(k);
          if (id < 0) continue;
          const Item it = item_at<NT>(P, pre, id);
          if (it.n == 0) continue;
          if (c > 0) ok = mbar_wait(q_free, (c - 1) & 1, P.err);
          if (!ok) break;
          ++c;
          const int nt = it.rows > P.PT ? NT : 1;
          *info = make_int4(it.n, nt, it.base(it.n - 1) + BN - it.nk, 0);
          mbar_arrive_expect_tx(q_full, (uint32_t)(nt * used * D * 2));
          for (int t = 0; t < nt; ++t)
#pragma unroll
            for (int g = 0; g < D / 64; ++g)
              tma_load_4d(qs + t * C::QBYTES + g * ROWS * 128, &mapQ, 0, it.h * P.G, it.q0 + t * P.PT, g, q_full);
        }
        if (ok && c > 0) ok = mbar_wait(q_free, (c - 1) & 1, P.err);
        if (ok) {  // no item is left
          *info = make_int4(0, 0, 0, 0);
          mbar_arrive(q_full);
        } else if (c > 0) {
          mbar_wait(q_full, (c - 1) & 1, P.err);
        }
      }
      __syncwarp();
    } else if (warp == C::SOFT) {
      // ------------------------------------------------- MMA issuer --
      constexpr uint32_t IDS = tc::idesc_bf16_f32(ROWS, BN, false);
      constexpr uint32_t IDO = tc::idesc_bf16_f32(ROWS, D, true);
      // descriptors: queries and keys K-major, values with rows along K
      const uint64_t dq = tc::smem_desc_sw128(smem_u32(qs), 16, 1024), dk = tc::smem_desc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_u32(ring + NK * SLOT), VK * 128, 1024);
      const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32), k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32);
      const uint32_t v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
      const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
      const bool leader = tc::elect_one();
      // After a wait that ran out the warp goes through the rest of the item
      // without waiting or issuing, so that its lanes stay together.
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = spin_wait(bar, parity, P.err);
      };
      struct Cursor {  // a ring's next slot
        int slot;
        uint32_t parity;
        __device__ __forceinline__ void step(int slots) {
          if (++slot == slots) {
            slot = 0;
            parity ^= 1;
          }
        }
      };
      Cursor ck{0, 0}, cv{0, 0};
      uint32_t c = 0;                     // items with work so far
      uint32_t sj[NT] = {}, pj[NT] = {};  // blocks of each tile: S issued, P consumed
      uint32_t oc[NT] = {};               // items of each tile
      while (ok) {
        wait(q_full, c & 1);
        // (a limit may run out in some lanes while the phase completes for others)
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++c;
        // n blocks, nt tiles; the last block's rows past the sequence's keys
        const int n = __shfl_sync(0xffffffffu, info->x, 0), nt = __shfl_sync(0xffffffffu, info->y, 0);
        const int beyond = __shfl_sync(0xffffffffu, info->z, 0);
        if (n == 0) break;
        // S of the next block for tiles ta..tb1-1; `release`: they are its last
        auto issue_s = [&](int ta, int tb1, bool release, bool last) {
          Cursor at = ck;
#pragma unroll
          for (int x = 0; x < PARTS; ++x) {
            if (ta == 0) wait(&full[at.slot], at.parity);  // (tile 1 follows tile 0)
            tc::fence_after_sync();
            if (leader && ok) {
              const uint32_t ka = k_lo + at.slot * (SLOT / 16);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (t < ta || t >= tb1) continue;
                const uint32_t sb = NSB == 2 ? (sj[0] & 1) : (uint32_t)t;
#pragma unroll
                for (int ks = 0; ks < KG * 4; ++ks)
                  tc::mma_bf16(tb + C::TS + sb * BN,
                               q_lo + (t * C::QBYTES + (x * KG + (ks >> 2)) * ROWS * 128 + (ks & 3) * 32) / 16, q_hi,
                               ka + ((ks >> 2) * BN * 128 + (ks & 3) * 32) / 16, k_hi, IDS,
                               (x > 0 || ks > 0) ? 1u : 0u);
                if (x == PARTS - 1) tc::commit(&s_full[sb]);
              }
              if (release) tc::commit(&empty[at.slot]);
              if (last && x == PARTS - 1) tc::commit(q_free);
            }
            at.step(NK);
          }
          if (release) ck = at;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (t >= ta && t < tb1) ++sj[t];
        };
        issue_s(0, nt, true, n == 1);
        for (int j = 0; j < n; ++j) {
          const bool more = j + 1 < n;
          if (NSB == 2 && more) issue_s(0, 1, true, j + 2 == n);  // runs during this block's softmax
          // rows past the sequence's keys belong to others: they count as zero
          const int past = more ? 0 : beyond;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t >= nt) continue;
            const uint32_t sb = NSB == 2 ? (pj[t] & 1) : (uint32_t)t;
            if (j == 0 && oc[t] > 0) wait(&o_free[t], (oc[t] - 1) & 1);
            if (NSB == 2) wait(&p_full[sb], (pj[t] >> 1) & 1);
            Cursor at = cv;
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              if (t == 0) wait(&full[5 + at.slot], at.parity);
              // keys of this slot that are the sequence's; the rest of their piece
              // belongs to others and counts as zero, later rows are old values
              const int kept = VK - imax(0, past - (PARTS - 1 - x) * VK);
              if (kept > 0 && kept % PIECE != 0 && t == 0) {
                uint8_t *vb = ring + (NK + at.slot) * SLOT;
                for (int y = lane; y < (PIECE - kept % PIECE) * (D / 8); y += 32) {
                  const int r = kept + y / (D / 8), z = y % (D / 8);
                  *reinterpret_cast<uint4 *>(vb + (z >> 3) * VK * 128 + r * 128 + (z & 7) * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
              }
              // one S buffer: the first half of the keys while the second's P is made
              constexpr int STEPS = NSB == 1 ? 2 : 1;
#pragma unroll
              for (int y = 0; y < STEPS; ++y) {
                if (NSB == 1) wait(y == 0 ? &p_half[sb] : &p_full[sb], pj[t] & 1);
                tc::fence_after_sync();
                if (leader && ok) {
                  const uint32_t va = v_lo + at.slot * (SLOT / 16);
#pragma unroll
                  for (int ks = y * (VK / 16 / STEPS); ks < (y + 1) * (VK / 16 / STEPS); ++ks)
                    tc::mma_bf16_ts(tb + C::TO + t * D, tb + C::TS + sb * BN + (x * (VK / 16) + ks) * 8,
                                    va + ks * 2048 / 16, v_hi, IDO, (x > 0 || ks > 0) ? 1u : (uint32_t)j);
                }
              }
              if (leader && ok) {
                if (x == PARTS - 1) tc::commit(&o_done[sb]);
                if (t == nt - 1) tc::commit(&empty[5 + at.slot]);
              }
              at.step(NV);
            }
            if (t == nt - 1) cv = at;
            ++pj[t];
            if (NSB == 1 && more) issue_s(t, t + 1, t == nt - 1, t == nt - 1 && j + 2 == n);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (t < nt) ++oc[t];
        ok = __all_sync(0xffffffffu, ok);
      }
      if (leader) {  // every product issued above has completed before TMEM is released
        tc::commit(idle);
        spin_wait(idle, 0, P.err);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------ softmax --
    setmaxnreg_inc<216>();
    constexpr int HALVES = C::HALVES, COLS = BN / HALVES;  // keys of a block that are this thread's
    const int t = HALVES == 1 ? warp >> 2 : 0;  // tile
    const int hf = HALVES == 1 ? 0 : warp >> 2;  // half of a block's keys, and of O's columns
    const int r = (warp & 3) * 32 + lane;       // row = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int ir = r / P.G;                     // position in the tile
    const float sl2e = P.sl2e;
    const f2 scale2 = pack2(sl2e, sl2e);
    const uint32_t tO = tbase + C::TO + t * D + lane_off;
    constexpr int O0 = D / HALVES;
    bool ok = true;
    uint32_t cnt = 0;  // blocks of this tile so far
    // The second product of the latest block.  The barrier's phase before it
    // is known to be over: its S (one S buffer: S of the latest block) was
    // issued after that product.
    auto wait_product = [&]() {
      const uint32_t at = cnt - 1;
      if (ok) ok = spin_wait(&o_done[NSB == 2 ? (at & 1) : (uint32_t)t], (NSB == 2 ? at >> 1 : at) & 1, P.err);
      ok = __all_sync(0xffffffffu, ok);
    };
    // The two halves of a row trade a value; slots alternate, so that one
    // barrier a trade is enough.
    uint32_t trades = 0;
    auto trade = [&](float x) {
      float *at = xchg + (trades & 1) * 2 * ROWS;
      ++trades;
      at[hf * ROWS + r] = x;
      named_barrier(2 + (warp & 3), 64);
      return at[(hf ^ 1) * ROWS + r];
    };
    int id = rounds > 0 ? item_id(0) : -1;
    Item it{};
    if (id >= 0) it = item_at<NT>(P, pre, id);
    for (int k = 0; k < rounds; ++k) {
      if (id < 0 || (t > 0 && it.rows <= P.PT)) {  // nothing for this tile
        if (k + 1 < rounds) {
          id = item_id(k + 1);
          if (id >= 0) it = item_at<NT>(P, pre, id);
        }
        continue;
      }
      const bool mine = ir < P.PT && t * P.PT + ir < it.rows;  // a row of the prompt
      const int pt = it.p0 + t * P.PT, p = pt + ir;            // position of the tile's first row, of this one
      const int plast = it.p0 + imin(it.rows, (t + 1) * P.PT) - 1;
      float m = -INFINITY, l = 0.f;
      // Both halves of a row take part in every trade whatever `ok` says (the
      // barriers have no time limit); after a wait that ran out only the work
      // is skipped.
      for (int j = 0; j < it.n; ++j, ++cnt) {
        const uint32_t sb = NSB == 2 ? (cnt & 1) : (uint32_t)t;
        const uint32_t tS = tbase + C::TS + sb * BN + hf * COLS + lane_off;
        if (ok) ok = spin_wait(&s_full[sb], (NSB == 2 ? cnt >> 1 : cnt) & 1, P.err);
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        uint32_t raw[COLS / 32][32];
        if (ok) {
#pragma unroll
          for (int c = 0; c < COLS / 32; ++c) tc::ld32(tS + 32 * c, raw[c]);
          tc::wait_ld();
        }
        const int base = it.base(j);
        if (base + BN - 1 > pt || (P.window > 0 && base <= plast - P.window && base + BN > P.sinks)) {
          // key c of the block is seen iff c <= hi and (c > lo or c < sk)
          const int at = base + hf * COLS, hi = p - at, lo = P.window > 0 ? hi - P.window : -1;
          const int sk = P.sinks - (j == 0 && it.ns == 0 ? hf * COLS : at);
#pragma unroll
          for (int c = 0; c < COLS / 32; ++c) {
            auto below = [&](int n) {  // bits 0..n-1 of this group of 32
              const int b = n - 32 * c;
              return b <= 0 ? 0u : b >= 32 ? 0xFFFFFFFFu : (1u << b) - 1u;
            };
            const uint32_t seen = below(hi + 1) & (~below(lo + 1) | below(sk));
#pragma unroll
            for (int e = 0; e < 32; ++e) raw[c][e] = (seen >> e & 1u) ? raw[c][e] : 0xFF800000u;  // -inf
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx4[i] = max3(mx4[i], __uint_as_float(raw[c][e + i]), __uint_as_float(raw[c][e + 4 + i]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        if (HALVES == 2) mx = fmaxf(mx, trade(mx));
        mx *= sl2e;
        float alpha = 1.f;
        if (mx > m + RESCALE) {
          alpha = m == -INFINITY ? 0.f : ex2_approx(m - mx);
          m = mx;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // the previous block's product is in O before it is rescaled
          wait_product();
          tc::fence_after_sync();
          if (ok) {
#pragma unroll 1
            for (int c0 = hf * O0; c0 < (hf + 1) * O0; c0 += 32) {
              uint32_t o[32];
              tc::ld32(tO + c0, o);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tc::st32(tO + c0, o);
            }
            tc::wait_st();
          }
          l *= alpha;
        }
        const float nb = m == -INFINITY ? 0.f : -m;
        const f2 nbase = pack2(nb, nb);
        f2 sum0 = 0, sum1 = 0;
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = unpack2(fma2(pack2(__uint_as_float(raw[c][2 * e]), __uint_as_float(raw[c][2 * e + 1])),
                                          scale2, nbase));
            const float y0 = ex2_approx(x.x), y1 = ex2_approx(x.y);
            if (e & 1)
              sum1 = add2(sum1, pack2(y0, y1));
            else
              sum0 = add2(sum0, pack2(y0, y1));
            pk[e] = pack_bf16x2(y0, y1);
          }
          // over S columns that both halves have read: this half's P follows the other's
          if (ok) tc::st16(tbase + C::TS + sb * BN + (hf * COLS) / 2 + 16 * c + lane_off, pk);
          if (NSB == 1 && c == COLS / 64 - 1) {
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[sb]);
          }
        }
        const float2 s2 = unpack2(add2(sum0, sum1));
        l += s2.x + s2.y;
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
      }
      const Item now = it;
      if (k + 1 < rounds) {  // the next item is looked up while the last product runs
        id = item_id(k + 1);
        if (id >= 0) it = item_at<NT>(P, pre, id);
      }
      if (now.n > 0) {
        wait_product();
        tc::fence_after_sync();
      }
      if (HALVES == 2) l += trade(l);
      // O / l to bf16.  Read so that the lanes of a quad hold neighbouring
      // columns of a row; four quad lanes then trade 4-byte pieces for 16
      // consecutive bytes each, and a store covers eight rows' 64 bytes (one
      // row a lane would take 32 sectors a store).
      constexpr int NG = O0 / 64;
      const float f = l != 0.f ? 1.f / l : 0.f;
      const long long at = (mine && ok) ? (long long)(now.q0 + t * P.PT + ir) * P.o.token_stride +
                                              (long long)(now.h * P.G + r - ir * P.G) * P.o.head_stride + hf * O0
                                        : -1LL;
      const int tq = lane & 3;
#pragma unroll 1
      for (int x0 = 0; x0 < 2 * NG; ++x0) {  // 16 rows of 64 columns at a time
        const int lh = x0 / NG, c = x0 % NG;
        uint32_t o[32];
        if (now.n > 0) {
          if (ok) {
            tc::ld_16x64(tbase + C::TO + t * D + ((uint32_t)((warp & 3) * 32 + 16 * lh) << 16) + hf * O0 + 64 * c, o);
            tc::wait_ld();
          }
          if (x0 == 2 * NG - 1) {  // O is read out
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[t]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 16 * lh + 8 * i + (lane >> 2);
          const float fr = __shfl_sync(0xffffffffu, f, row);
          const long long to = __shfl_sync(0xffffffffu, at, row);
          __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(P.o.ptr) + to + 64 * c + 8 * tq;
          const f2 fr2 = pack2(fr, fr);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int y = 16 * g + 4 * e + 2 * i;
              const float2 z = unpack2(mul2(pack2(__uint_as_float(o[y]), __uint_as_float(o[y + 1])), fr2));
              x[e] = pack_bf16x2(z.x, z.y);
            }
            auto trade4 = [&](uint32_t &lo, uint32_t &hi, int bit) {
              const bool up = tq & bit;
              const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
              if (up) lo = y; else hi = y;
            };
            trade4(x[0], x[1], 1);
            trade4(x[2], x[3], 1);
            trade4(x[0], x[2], 2);
            trade4(x[1], x[3], 2);
            // no key seen: zeros, whatever O holds
            const uint4 v = fr != 0.f ? make_uint4(x[0], x[1], x[2], x[3]) : make_uint4(0u, 0u, 0u, 0u);
            if (to >= 0) *reinterpret_cast<uint4 *>(out + 32 * g) = v;
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::SOFT) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512u);
  }
}

// 4-D map of rows [T][H][D]: keys and values (column, token, 64-column group,
// head) in boxes of 64 x b1 x b2, queries (column, head, token, group) in
// boxes of 64 x b1 x b2; 128-byte swizzle, zeros past the last token.
// `any`: an address to stand in for that of no rows.
static bool make_map(CUtensorMap *map, const sv_rows *r, int T, int H, int D, bool query, int b1, int b2, void *any) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  const cuuint64_t t = (cuuint64_t)imax(T, 1), g = (cuuint64_t)(D / 64);
  // the stride of a dimension of one is never used, but has to be a valid one
  const cuuint64_t ts = T > 1 ? (cuuint64_t)r->token_stride * 2 : 128, hs = H > 1 ? (cuuint64_t)r->head_stride * 2 : 128;
  cuuint64_t dk[4] = {64, t, g, (cuuint64_t)H}, sk[3] = {ts, 128, hs};
  cuuint64_t dq[4] = {64, (cuuint64_t)H, t, g}, sq[3] = {hs, ts, 128};
  cuuint32_t bk[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, bq[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, T > 0 ? r->ptr : any, query ? dq : dk, query ? sq : sk, query ? bq : bk, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int TILES>
static sv_status run(const sv_rows *q, const sv_rows *k, const sv_rows *v, Params &P, int sms, cudaStream_t s) {
  using C = Cfg<D, TILES>;
  CUtensorMap mq, mk, mv, mkp, mvp;
  if (!make_map(&mq, q, P.Tq, P.Hkv * P.G, D, true, P.G, P.PT, q->ptr) ||
      !make_map(&mk, k, P.Tk, P.Hkv, D, false, BN, C::KG, q->ptr) ||
      !make_map(&mv, v, P.Tk, P.Hkv, D, false, C::VK, D / 64, q->ptr) ||
      !make_map(&mkp, k, P.Tk, P.Hkv, D, false, PIECE, 1, q->ptr) ||
      !make_map(&mvp, v, P.Tk, P.Hkv, D, false, PIECE, 1, q->ptr))
    return SV_ERR_CUDA;
  const size_t prefix = ((size_t)P.B + 1) * 4;
  P.by_span = (uint32_t)((0x100000000ull + P.PT * C::NT - 1) / (P.PT * C::NT) - (P.PT * C::NT == 1));
  P.few_slots = prefix <= HEADER - PREFIX ? 0 : 1;
  const size_t smem = C::RING + (P.few_slots ? 128 * 1024 + prefix : 160 * 1024);
  static_assert(C::RING + 160 * 1024 <= 227 * 1024 && C::RING + 128 * 1024 + (MAX_B + 1) * 4 <= 227 * 1024, "shared memory");
  // at most one item more per sequence than the rows fill
  P.most = P.Tq / (P.PT * C::NT) + P.B;
  const long long items = (long long)P.most * P.Hkv;
  const int ctas = (int)lmin(items, sms);
  return from_cuda(launch_early(window_kernel<D, TILES>, dim3(ctas), dim3(C::THREADS), smem, s, mq, mk, mv,
                                mkp, mvp, P));
}

static sv_status run_any(const sv_rows *q, const sv_rows *k, const sv_rows *v, Params &P, int D, int sms,
                         cudaStream_t s) {
  if (D == 256) return run<256, 1>(q, k, v, P, sms, s);
  // Two tiles a CTA use the tensor cores best (8192 rows of 32 heads, causal:
  // 357 us against 425), but their items are twice as long: with fewer than two
  // for every SM single tiles fill the GPU more evenly (seven prompts of 2 to
  // 901 rows: 20 us against 25; four of 519 to 1200: 35 against 30).
  const long long pairs = ((long long)P.Tq / (P.PT * 2) + P.B) * P.Hkv;
  return pairs >= 2 * sms ? run<128, 2>(q, k, v, P, sms, s) : run<128, 1>(q, k, v, P, sms, s);
}

}  // namespace window
}  // namespace sv

using namespace sv;

extern "C" {

size_t window_attn_workspace_bytes(int B, int Hq, int Hkv, int D) {
  (void)B, (void)Hq, (void)Hkv, (void)D;
  return 0;
}

sv_status window_attn(const sv_rows *q, const sv_rows *k, const sv_rows *v, const sv_rows *o,
                      const int32_t *cu_q, const int32_t *cu_k, int B, int Tq, int Tk, int Hq, int Hkv, int D,
                      float scale, int window, int sinks, void *workspace, size_t ws_bytes, sv_stream_t stream) {
  (void)workspace, (void)ws_bytes;
  if (B < 0 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1 || D < 1 || Hq % Hkv != 0) return SV_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return SV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return SV_ERR_INVALID_ARG;
  if (D != 128 && D != 256) return SV_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G > window::ROWS || B > window::MAX_B) return SV_ERR_UNSUPPORTED;
  if (Tq > 0x40000000 || Tk > 0x40000000 || window > 0x40000000) return SV_ERR_UNSUPPORTED;
  for (const sv_rows *r : {q, o})
    if (!paged::good_rows(r, Tq)) return SV_ERR_INVALID_ARG;
  for (const sv_rows *r : {k, v})
    if (!paged::good_rows(r, Tk)) return SV_ERR_INVALID_ARG;
  if (B > 0 && (!cu_q || !cu_k)) return SV_ERR_INVALID_ARG;
  if (!paged::aligned(cu_q, 4) || !paged::aligned(cu_k, 4)) return SV_ERR_INVALID_ARG;
  if (B == 0 || Tq == 0) return SV_OK;
  // a tensor map steps by every stride: rows that repeat (stride 0) have none
  if ((Tq > 1 && !q->token_stride) || (Hq > 1 && !q->head_stride)) return SV_ERR_UNSUPPORTED;
  for (const sv_rows *r : {k, v})
    if ((Tk > 1 && !r->token_stride) || (Hkv > 1 && !r->head_stride)) return SV_ERR_UNSUPPORTED;
  // the items of all KV heads, and the places of a round behind them, are counted in 31 bits
  const int pt = window::ROWS / G;
  if (((long long)Tq / pt + B) * Hkv > 0x7fff0000LL) return SV_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return SV_ERR_CUDA;
  window::Params P{};
  P.o = *o;
  P.cu_q = cu_q;
  P.cu_k = cu_k;
  P.err = device_error_word();
  if (!P.err) return SV_ERR_CUDA;
  P.B = B;
  P.Tq = Tq;
  P.Tk = Tk;
  P.Hkv = Hkv;
  P.G = G;
  P.PT = pt;
  P.sl2e = scale * 1.4426950408889634f;
  P.window = window;
  P.sinks = sinks;
  P.stall = launch_flags() & SV_LAUNCH_TEST_STALL_COPY ? 1 : 0;
  return window::run_any(q, k, v, P, D, sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
