// gdn_step.cu -- the gated delta rule token by token, for many sequences over
// a pool of states: one new token each, or the rows of a verify step behind
// what each accepted of its last one.
//
// Per value head (key head h / (Hv/Hk)) the state S is dv x dk, and a token
// makes   S <- a S + u k^T,  u = b (v - a S k),  a = exp(g),  and reads o = S q.
//
// What bounds it: a state is read once and written once (8 * dk * dv bytes a
// value head) and meets few tokens, so HBM; for one sequence the chain of a
// token's two dot products.  Rows of S are independent under the rule: eight
// lanes hold one in registers for the whole call (lane `sub` columns
// 4*sub + 32*j .. +3, so that the eight read whole 128-byte lines and their
// shared reads of a key meet no bank twice), a dot product ends in three
// shuffles, and a block is a few rows of one head.  The state's loads are
// issued before the tokens are staged (fp32, in shared memory), so both wait
// for memory together.
#include "gdn_pool.cuh"

namespace sv {
namespace gdn {
namespace {

constexpr int LPR = 8;         // lanes per state row
constexpr int MAX_STAGE = 32;  // tokens staged at a time

// Sum over the eight lanes of a row.
__device__ __forceinline__ float over_row(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int NJ>
__device__ __forceinline__ float dot_row(const f2 (&row)[2 * NJ], const float *x) {
  f2 s[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(x + 32 * j);
    s[0] = fma2(row[2 * j], y.x, s[0]);
    s[1] = fma2(row[2 * j + 1], y.y, s[1]);
  }
  const float2 z = unpack2(add2(s[0], s[1]));
  return over_row(z.x + z.y);
}

// Stages n bf16 rows of DK (head `h`, from row `r0` on) as fp32.
template <int DK>
__device__ __forceinline__ void stage_rows(float *dst, const sv_rows &src, long long r0, int h, int n) {
  const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(src.ptr) + (long long)h * src.head_stride;
  for (int e = threadIdx.x; e < n * (DK / 8); e += blockDim.x) {
    const int t = e / (DK / 8), c = e % (DK / 8);
    const uint4 w = *reinterpret_cast<const uint4 *>(p + (r0 + t) * src.token_stride + c * 8);
    float4 *d = reinterpret_cast<float4 *>(dst + (size_t)e * 8);
    d[0] = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
    d[1] = make_float4(bf16lo(w.z), bf16hi(w.z), bf16lo(w.w), bf16hi(w.w));
  }
}

template <int DK>
__global__ void __launch_bounds__(256, DK <= 128 ? 6 : 4) tokens_kernel(const __grid_constant__ PoolParams P) {
  constexpr int NJ = DK / 32;
  extern __shared__ __align__(16) float sm[];
  const int rows = blockDim.x / LPR;
  const int i0 = blockIdx.x * rows, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (P.Hv / P.Hk);
  const int tid = threadIdx.x, r = tid / LPR, sub = tid % LPR, i = i0 + r;
  const bool live = i < P.dv, report = blockIdx.x == 0 && h == 0 && tid == 0;
  float *sk = sm, *sq = sk + P.stage * DK, *sv_ = sq + P.stage * DK, *sab = sv_ + P.stage * rows;
  pdl_wait();
  const int slot = slot_of(P, b, report);
  const int2 own = rows_of(P, b, report);
  int replay = 0;
  if (P.n_replay) {
    replay = P.n_replay[b];
    if (replay < 0 || replay > P.tape_M) {
      if (report) atomicOr(P.err, ERR_INDEX);
      replay = imin(imax(replay, 0), P.tape_M);
    }
  }
  const bool kept = slot >= 0 && live;
  float *srow = P.states.ptr + (slot >= 0 ? slot : 0) * P.states.slot_stride + ((long long)h * P.dv + (live ? i : 0)) * DK + sub * 4;
  f2 row[2 * NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    ulonglong2 x = make_ulonglong2(0, 0);
    if (kept) x = *reinterpret_cast<const ulonglong2 *>(srow + 32 * j);
    row[2 * j] = x.x, row[2 * j + 1] = x.y;
  }
  auto keep = [&]() {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (kept) *reinterpret_cast<ulonglong2 *>(srow + 32 * j) = make_ulonglong2(row[2 * j], row[2 * j + 1]);
  };
  // the tape's tokens, then the sequence's own
  for (int part = 0; part < 2; ++part) {
    const bool mine = part == 1;
    const int n = mine ? own.y : replay;
    const long long r0 = mine ? own.x : (long long)b * P.tape_M;
    const sv_rows &K = mine ? P.k : P.tk, &V = mine ? P.v : P.tv;
    const float *G = mine ? P.g : P.tg, *Bt = mine ? P.b : P.tb;
    for (int t0 = 0; t0 < n; t0 += P.stage) {
      const int m = imin(P.stage, n - t0);
      if (part + t0 > 0) __syncthreads();  // what was staged has been read
      stage_rows<DK>(sk, K, r0 + t0, hk, m);
      if (mine) stage_rows<DK>(sq, P.q, r0 + t0, hk, m);
      for (int e = tid; e < m * rows; e += blockDim.x) {
        const int t = e / rows, x = e % rows;
        sv_[e] = i0 + x < P.dv ? __bfloat162float(static_cast<const __nv_bfloat16 *>(
                                     V.ptr)[(r0 + t0 + t) * V.token_stride + h * V.head_stride + i0 + x])
                               : 0.f;
      }
      for (int t = tid; t < m; t += blockDim.x) {
        sab[2 * t] = expf(G[(r0 + t0 + t) * P.Hv + h]);
        sab[2 * t + 1] = Bt[(r0 + t0 + t) * P.Hv + h];
      }
      __syncthreads();
      for (int t = 0; t < m; ++t) {
        const float *kk = sk + t * DK + sub * 4;
        const float a = sab[2 * t];
        const float u = sab[2 * t + 1] * (sv_[t * rows + r] - a * dot_row<NJ>(row, kk));
        const f2 a2 = pack2(a, a), u2 = pack2(u, u);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(kk + 32 * j);
          row[2 * j] = fma2(a2, row[2 * j], mul2(u2, y.x));
          row[2 * j + 1] = fma2(a2, row[2 * j + 1], mul2(u2, y.y));
        }
        if (mine) {
          const float ov = dot_row<NJ>(row, sq + t * DK + sub * 4);
          if (sub == 0 && live) {
            const long long at = (r0 + t0 + t) * P.o.token_stride + h * P.o.head_stride + i;
            if (P.o_f32)
              static_cast<float *>(P.o.ptr)[at] = ov;
            else
              static_cast<__nv_bfloat16 *>(P.o.ptr)[at] = __float2bfloat16_rn(ov);
          }
        }
      }
    }
    // (a state that no token has changed is not written)
    if (mine ? P.commit && own.y + replay > 0 : !P.commit && replay > 0) keep();
  }
}

// ---- many states: a stream of tiles through shared memory ----
constexpr int TOKENS = 16;  // tokens of a sequence (tape and own) at most
// Shared memory a block: two share an SM's 228 KB, of which a block takes 1 KB itself.
constexpr int STREAM_BYTES = 115200;
constexpr int WORK_WARPS = 8, STREAM_THREADS = (WORK_WARPS + 2) * 32;

// RP: rows of a thread.
template <int DK, int RP>
struct SL {
  static constexpr int TILE = RP * WORK_WARPS * 32 / LPR;
  static constexpr int STATE = TILE * DK * 4;
  // of a stage: the rows of S, the tokens' gates (a, b), what the tile is, the tokens
  static constexpr int GATES = STATE, META = GATES + TOKENS * 8, TOKEN = META + 32;
  static constexpr int EACH = 4 * DK + 2 * TILE;  // bytes of a token: key, query, values
  __host__ __device__ static int stage(int tokens) { return (TOKEN + tokens * EACH + 127) / 128 * 128; }
};

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The same rule on the same lanes.  What differs: a block walks over tiles (sequence, head, 32 or
// 64 rows), one warp asking for the next ones' states, keys, queries and values by bulk copies, one
// writing the states back; as many bytes are on their way as the ring holds, whatever the
// tiles' own latency (48 heads of 128 x 128: one token of 61 sequences 79 us with a block a tile, 60 this
// way, 6.5 TB/s; 24 sequences of 4 rows behind 2 replayed on average 53 and 36, the rows' instructions).
template <int DK, int RP>
__global__ void __launch_bounds__(STREAM_THREADS, 2) stream_kernel(const __grid_constant__ PoolParams P, int stages, int tiles, int row_tiles) {
  using Y = SL<DK, RP>;
  constexpr int NJ = DK / 32, TILE = Y::TILE;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[16], done[16], empty[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tape = P.tape_M, tokens = tape + P.M, size = Y::stage(tokens);
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], WORK_WARPS);
      mbar_init(&empty[i], 1);
    }
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  // (tiles may be next to 2^31)
  const int mine = tiles > (int)blockIdx.x ? (tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  // sequence, head and first row of this block's k-th tile
  struct Where {
    int b, h, i0;
  };
  auto where = [&](int k) {
    const int t = blockIdx.x + k * gridDim.x, x = t / row_tiles, b = x / P.Hv;
    return Where{b, x - b * P.Hv, (t - x * row_tiles) * TILE};
  };
  bool ok = true;
  if (warp == WORK_WARPS) {
    // ------------------------------------------------------------ copies in --
    struct Ask {  // of a tile, asked for one tile ahead
      Where w;
      int slot, replay;
      float g, b;  // of token `lane`
    };
    auto ask = [&](int k) {
      Ask a{};
      a.w = where(k);
      a.slot = P.slots[a.w.b];
      a.replay = P.n_replay ? P.n_replay[a.w.b] : 0;
      if (lane < tokens) {
        const bool own = lane >= tape;
        const long long at = (own ? (long long)a.w.b * P.M + lane - tape : (long long)a.w.b * tape + lane) * P.Hv + a.w.h;
        a.g = own ? P.g[at] : P.tg[at];
        a.b = own ? P.b[at] : P.tb[at];
      }
      return a;
    };
    Ask next{};
    if (mine > 0) next = ask(0);
    for (int k = 0; k < mine && ok; ++k) {
      Ask a = next;
      if (k + 1 < mine) next = ask(k + 1);
      const int st = k % stages;
      if (k >= stages && lane == 0) ok = mbar_wait(&empty[st], (k / stages - 1) & 1, P.err);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      uint8_t *at = ring + st * size;
      if (a.slot >= P.states.num_slots || a.replay < 0 || a.replay > tape) {
        if (lane == 0) atomicOr(P.err, ERR_INDEX);
        a.slot = a.slot >= P.states.num_slots ? -1 : a.slot;
        a.replay = imin(imax(a.replay, 0), tape);
      }
      if (lane < tokens) *reinterpret_cast<float2 *>(at + Y::GATES + lane * 8) = make_float2(expf(a.g), a.b);
      if (lane == 0) {
        *reinterpret_cast<int4 *>(at + Y::META) = make_int4(a.slot, a.replay, a.w.b, a.w.h);
        *reinterpret_cast<int *>(at + Y::META + 16) = a.w.i0;
      }
      __syncwarp();
      const int rows = imin(TILE, P.dv - a.w.i0);
      const uint32_t state = a.slot >= 0 ? rows * DK * 4 : 0, values = rows * 2;
      if (lane == 0)
        mbar_arrive_expect_tx(&full[st], state + a.replay * (DK * 2 + values) + P.M * (DK * 4 + values));
      __syncwarp();
      const int hk = a.w.h / (P.Hv / P.Hk);
      if (lane == 31 && state)
        bulk_load(at, P.states.ptr + a.slot * P.states.slot_stride + ((long long)a.w.h * P.dv + a.w.i0) * DK, state, &full[st]);
      if (lane < tape ? lane < a.replay : lane < tokens) {
        const bool own = lane >= tape;
        const long long t = own ? (long long)a.w.b * P.M + lane - tape : (long long)a.w.b * tape + lane;
        const sv_rows &K = own ? P.k : P.tk, &V = own ? P.v : P.tv;
        uint8_t *to = at + Y::TOKEN + lane * Y::EACH;
        bulk_load(to, static_cast<const __nv_bfloat16 *>(K.ptr) + t * K.token_stride + hk * K.head_stride, DK * 2, &full[st]);
        if (own) bulk_load(to + DK * 2, static_cast<const __nv_bfloat16 *>(P.q.ptr) + t * P.q.token_stride + hk * P.q.head_stride, DK * 2, &full[st]);
        bulk_load(to + DK * 4, static_cast<const __nv_bfloat16 *>(V.ptr) + t * V.token_stride + a.w.h * V.head_stride + a.w.i0, values, &full[st]);
      }
      __syncwarp();
    }
  } else if (warp == WORK_WARPS + 1) {
    // ----------------------------------------------------------- states out --
    if (lane == 0) {
      int k = 0;
      for (; k < mine; ++k) {
        const int st = k % stages;
        if (!mbar_wait(&done[st], (k / stages) & 1, P.err)) break;
        uint8_t *at = ring + st * size;
        const int4 meta = *reinterpret_cast<const int4 *>(at + Y::META);
        const int i0 = *reinterpret_cast<const int *>(at + Y::META + 16);
        if (meta.x >= 0 && (meta.y > 0 || (P.commit && P.M > 0)))
          bulk_store(P.states.ptr + meta.x * P.states.slot_stride + ((long long)meta.w * P.dv + i0) * DK, at, imin(TILE, P.dv - i0) * DK * 4);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        // the tile before this one has been read out
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        if (k > 0) mbar_arrive(&empty[(k - 1) % stages]);
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      if (k == mine && k > 0) mbar_arrive(&empty[(k - 1) % stages]);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- rows --
    const int r = tid / LPR, sub = tid % LPR;
    for (int k = 0; k < mine; ++k) {
      const int st = k % stages;
      if (ok) ok = mbar_wait(&full[st], (k / stages) & 1, P.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t *at = ring + st * size;
      const int4 meta = *reinterpret_cast<const int4 *>(at + Y::META);
      const Where w{meta.z, meta.w, *reinterpret_cast<const int *>(at + Y::META + 16)};
      float *srow = reinterpret_cast<float *>(at) + r * DK + sub * 4;  // (rows of a thread: 32 apart)
      f2 row[RP][2 * NJ];
#pragma unroll
      for (int p = 0; p < RP; ++p)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const bool live = w.i0 + r + 32 * p < P.dv;
          const ulonglong2 x = meta.x >= 0 && live ? *reinterpret_cast<const ulonglong2 *>(srow + 32 * p * DK + 32 * j) : make_ulonglong2(0, 0);
          row[p][2 * j] = x.x, row[p][2 * j + 1] = x.y;
        }
      auto keep = [&]() {
#pragma unroll
        for (int p = 0; p < RP; ++p)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            *reinterpret_cast<ulonglong2 *>(srow + 32 * p * DK + 32 * j) = make_ulonglong2(row[p][2 * j], row[p][2 * j + 1]);
      };
      // this lane's pieces of a row of bf16
      auto pieces = [&](const uint8_t *x, f2 (&y)[2 * NJ]) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const uint2 z = *reinterpret_cast<const uint2 *>(x + sub * 8 + 64 * j);
          y[2 * j] = pack2(bf16lo(z.x), bf16hi(z.x)), y[2 * j + 1] = pack2(bf16lo(z.y), bf16hi(z.y));
        }
      };
      auto parts = [&](const f2 (&x)[2 * NJ], float (&out)[RP]) {
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          f2 s[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 2 * NJ; ++j) s[j & 1] = fma2(row[p][j], x[j], s[j & 1]);
          const float2 z = unpack2(add2(s[0], s[1]));
          out[p] = z.x + z.y;
        }
      };
      auto dots = [&](const f2 (&x)[2 * NJ], float (&out)[RP]) {
        parts(x, out);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
          for (int p = 0; p < RP; ++p) out[p] += __shfl_xor_sync(0xffffffffu, out[p], off);
      };
      auto token = [&](int n) {
        const uint8_t *x = at + Y::TOKEN + n * Y::EACH;
        const float2 ab = *reinterpret_cast<const float2 *>(at + Y::GATES + n * 8);
        f2 key[2 * NJ];
        float d[RP];
        pieces(x, key);
        dots(key, d);
        const f2 a2 = pack2(ab.x, ab.x);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          // (rows past the head's last are not stored, whatever stands there)
          const float v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(x + DK * 4)[r + 32 * p]);
          const float u = ab.y * (v - ab.x * d[p]);
          const f2 u2 = pack2(u, u);
#pragma unroll
          for (int j = 0; j < 2 * NJ; ++j) row[p][j] = fma2(a2, row[p][j], mul2(u2, key[j]));
        }
      };
#pragma unroll 1
      for (int n = 0; n < meta.y; ++n) token(n);
      if (!P.commit && meta.y > 0) keep();
      // the row that this lane writes outputs of: of two, the second half of the lanes' second
      const int mine = w.i0 + r + (RP == 2 ? sub / (LPR / 2) * 32 : 0);
      const bool writes = sub % (LPR / RP) == 0 && mine < P.dv;
      long long o = (long long)w.b * P.M * P.o.token_stride + w.h * P.o.head_stride + mine;
#pragma unroll 1
      for (int n = 0; n < P.M; ++n, o += P.o.token_stride) {
        token(tape + n);
        f2 query[2 * NJ];
        float d[RP];
        pieces(at + Y::TOKEN + (tape + n) * Y::EACH + DK * 2, query);
        parts(query, d);
        float x = d[0];
        if (RP == 2) {  // each half of the lanes goes on with one row
          const bool second = sub >= LPR / 2;
          x = (second ? d[RP - 1] : d[0]) + __shfl_xor_sync(0xffffffffu, second ? d[0] : d[RP - 1], LPR / 2);
        }
#pragma unroll
        for (int off = LPR / 2 / RP; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (writes) {
          if (P.o_f32)
            static_cast<float *>(P.o.ptr)[o] = x;
          else
            static_cast<__nv_bfloat16 *>(P.o.ptr)[o] = __float2bfloat16_rn(x);
        }
      }
      if (P.commit) keep();
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&done[st]);
    }
  }
}

template <int DK, int RP>
sv_status run_stream(const PoolParams &P, int sms, cudaStream_t s) {
  using Y = SL<DK, RP>;
  const int row_tiles = (P.dv + Y::TILE - 1) / Y::TILE;
  const int size = Y::stage(P.tape_M + P.M), stages = imin(16, STREAM_BYTES / size);
  return from_cuda(launch_early(stream_kernel<DK, RP>, dim3(2 * sms), dim3(STREAM_THREADS), (size_t)stages * size, s, P, stages,
                                (int)((long long)P.B * P.Hv * row_tiles), row_tiles));
}

template <int DK>
sv_status run_tokens(PoolParams &P, cudaStream_t s) {
  const long long small = (long long)P.B * P.Hv * ((P.dv + 7) / 8);
  const int sms = device_sm_count();
  if (sms <= 0) return SV_ERR_CUDA;
  // Few tokens of many states are streamed (values in whole 16 bytes); it pays from some
  // tiles a block on.
  // Two rows a thread share what it reads of keys and queries: at 64 columns always (tiles of 16 KB), at 128
  // from two tokens on (32 KB; 24 sequences of 48 heads, 4 + 4 tokens 35 us against 43, 4 tokens 29 against
  // 37, two tokens of 61 sequences 43 against 63, but one token of them 64 against 60).
  constexpr int ONE = DK == 64 ? 2 : 1;
  const long long tiles = (long long)P.B * P.Hv * ((P.dv + SL<DK, ONE>::TILE - 1) / SL<DK, ONE>::TILE);
  if (!P.cu && P.tape_M + P.M <= TOKENS && P.dv % 8 == 0 && tiles >= 4LL * sms && tiles <= 0x7fffffffLL) {
    if (DK == 128 && P.tape_M + P.M >= 2) return run_stream<DK, DK == 128 ? 2 : ONE>(P, sms, s);
    return run_stream<DK, ONE>(P, sms, s);
  }
  // Otherwise a block a few rows: eight while that leaves each SM few of them (one sequence of
  // 48 heads: 768), 32 beyond, where what a block stages is shared by more rows.
  const int threads = small > 16LL * sms ? 256 : 64, rows = threads / LPR;
  const size_t smem = (size_t)P.stage * (2 * DK + rows + 2) * 4;
  return from_cuda(launch_early(tokens_kernel<DK>, dim3((P.dv + rows - 1) / rows, P.Hv, P.B), dim3(threads), smem, s, P));
}

}  // namespace

sv_status launch_tokens(PoolParams &P, int dk, cudaStream_t s) {
  const int most = P.cu ? P.T : imax(P.M, P.tape_M);
  P.stage = imax(1, imin(most, MAX_STAGE));
  switch (dk) {
    case 64: return run_tokens<64>(P, s);
    case 128: return run_tokens<128>(P, s);
    default: return run_tokens<256>(P, s);
  }
}

}  // namespace gdn
}  // namespace sv

using namespace sv;

extern "C" {

sv_status gdn_step(const sv_states *states, const int32_t *slots, const sv_rows *tape_k, const sv_rows *tape_v,
                   const float *tape_g, const float *tape_beta, const int32_t *n_replay, int tape_M, const sv_rows *q,
                   const sv_rows *k, const sv_rows *v, const float *g, const float *beta, const sv_rows *o,
                   sv_dtype o_dtype, int B, int M, int commit, int Hk, int Hv, int dk, int dv, sv_stream_t stream) {
  if (B < 0 || M < 0 || tape_M < 0 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || dk < 1 || dv < 1) return SV_ERR_INVALID_ARG;
  if (o_dtype != SV_BF16 && o_dtype != SV_F32) return SV_ERR_INVALID_ARG;
  if (dk != 64 && dk != 128 && dk != 256) return SV_ERR_UNSUPPORTED;
  if (M > 64 || tape_M > 64 || Hv > 65535 || B > gdn::MAX_POOL_B || dv > 65536) return SV_ERR_UNSUPPORTED;
  if (sv_status e = gdn::check_states(states, Hv, dk, dv)) return e;
  const bool tape = n_replay != nullptr && tape_M > 0, rows = M > 0;
  if (B > 0 && (!slots || !paged::aligned(slots, 4) || !paged::aligned(n_replay, 4))) return SV_ERR_INVALID_ARG;
  if (rows) {
    for (const sv_rows *r : {q, k, v, o})
      if (!paged::good_rows(r, (long long)B * M)) return SV_ERR_INVALID_ARG;
    if (B > 0 && (!g || !beta || !paged::aligned(g, 4) || !paged::aligned(beta, 4))) return SV_ERR_INVALID_ARG;
  }
  if (tape) {
    for (const sv_rows *r : {tape_k, tape_v})
      if (!paged::good_rows(r, (long long)B * tape_M)) return SV_ERR_INVALID_ARG;
    if (B > 0 && (!tape_g || !tape_beta || !paged::aligned(tape_g, 4) || !paged::aligned(tape_beta, 4)))
      return SV_ERR_INVALID_ARG;
  }
  if (B == 0 || (!rows && !tape)) return SV_OK;
  gdn::PoolParams P{};
  P.states = *states;
  P.slots = slots;
  if (tape) {
    P.tk = *tape_k, P.tv = *tape_v, P.tg = tape_g, P.tb = tape_beta;
    P.n_replay = n_replay, P.tape_M = tape_M;
  }
  if (rows) P.q = *q, P.k = *k, P.v = *v, P.o = *o, P.g = g, P.b = beta;
  P.err = device_error_word();
  if (!P.err) return SV_ERR_CUDA;
  P.B = B, P.M = M, P.T = B * M, P.Hk = Hk, P.Hv = Hv, P.dv = dv;
  P.commit = commit ? 1 : 0;
  P.o_f32 = o_dtype == SV_F32 ? 1 : 0;
  return gdn::launch_tokens(P, dk, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
