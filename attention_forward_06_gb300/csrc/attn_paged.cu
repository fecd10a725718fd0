// attn_paged.cu -- attention of each sequence's newest tokens over a paged key/value
// cache (attn_paged.h).  Bound by the bytes of K and V: a query token of G heads per kv
// head makes 4 G D operations of the 4 D bytes of a key, so up to some 280 rows (tokens x
// heads of a group) the cache's bytes take longer than the tensor cores.
//
// attn_tree_kernel: one persistent CTA per SM.  The work is a list of key tiles (128
// keys of one kv head) ordered by sequence, 128-row tile, kv head and tile;
// every CTA takes an equal, contiguous part of it, found from the lengths on the device
// (one warp sums the sequences' tiles), so the load is even whatever the lengths are and
// the host needs none of them.  The 128 rows are the tokens of a sequence times the G query
// heads of a kv head.  An item is the part of one (rows, kv head)'s tiles that a CTA holds;
// one that holds all of them writes O and LSE, otherwise it leaves a normalised fp32
// partial and its LSE in the workspace (at most two per CTA: the item it
// begins with and the item it ends with), which attn_tree_merge_kernel joins.
//
// Twelve warps:
//   warps 0-3    softmax, one thread per row, and the epilogue
//   warps 4-7    V tiles from bf16 to fp16 in place, rows past the sequence zeroed
//   warp  8      TMA producer: K and V pages into a ring of tile slots
//   warp  9      tcgen05 issuer and TMEM owner
//   warps 10-11  Q rows into one of two buffers
// TMEM: S of even steps [0,128), of odd steps [128,256), O [256, 256 + D); P (fp16) over
// the last 64 columns of its S.  The issuer runs S one step ahead:
//   S(0) | S(g+1) PV(g) | S(g+2) PV(g+1) | ...   across items,
// so S(g+1) is ready when the softmax has handed over P(g).
//
// Softmax as attn_fwd.cu's: exponentials in log2 units against a reference value m that
// all of a row's sums share.  Here every tile's max is taken (the time is there) and m is
// moved only when P would pass 2^15: it is set 6 below the tile's max, so P of
// the largest key starts at 2^6 and fp16 keeps keys down to 2^-20 of it in full precision,
// 2^-30 at all.  O is then scaled in TMEM after PV(g-1) has finished.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_paged.h"
#include "host_util.h"
#include "kv_host.h"
#include "ptx.cuh"

using namespace attn;

namespace {

constexpr int BM = 128;  // rows (tokens x heads of a group) per item
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint32_t kRegsLaunch = 168;   // 65536 / 384
constexpr uint32_t kRegsSoftmax = 232;  // a whole S row lives in registers
constexpr uint32_t kRegsConvert = 136;
constexpr uint32_t kRegsOther = 136;
static_assert(128 * (kRegsSoftmax + kRegsConvert + kRegsOther) <= kThreads * kRegsLaunch, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 2 * BN;
constexpr uint64_t kTimeoutNs = 4000000000ull;
constexpr uint64_t kDrainTimeoutNs = 500000000ull;
constexpr float kStart = 6.0f;   // log2 of P of the largest key when m is set
constexpr float kLimit = 15.0f;  // log2 of P at which m moves (fp16 holds up to 2^16)
constexpr int kMaxCtas = 192;    // partial slots are sized for this many CTAs
constexpr int kSeqSlots = 4;
constexpr int kSeqConsumers = 11;  // every warp but the producer

constexpr int kSiteProducer = 1, kSiteIssuer = 2, kSiteSoftmax = 3, kSiteConvert = 4, kSiteQuery = 5;
constexpr int kSiteInput = 100;  // lengths or page numbers that do not fit

template <int D>
struct Cfg {
  static constexpr int kTileBytes = BN * D * 2;
  static constexpr int kColBlockBytes = BN * 128;
  // slots of the K and of the V ring: 160 or 192 KB in flight.  S runs a step ahead of PV, so K is
  // needed earlier and held shorter
  static constexpr int kK = D == 128 ? 3 : 6;
  static constexpr int kV = D == 128 ? 2 : 6;
  static constexpr int kSmemBytes = (2 + kK + kV) * kTileBytes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

struct Params {
  const __nv_bfloat16* q;
  int64_t q_token, q_head;
  __nv_bfloat16* o;
  float* lse;
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  const uint32_t* mask;  // [tokens][mask_words] or null (a chain)
  int mask_words;
  int rows, max_pages, n_pages, page_size;  // rows: sequences
  int n_tokens, Hq, Hkv, G;
  int R;  // tokens per item: BM / G
  int window, sinks;
  float c;  // scale * log2(e)
  float* part_o;    // [kMaxCtas][2][BM][D]
  float* part_lse;  // [kMaxCtas][2][BM], log2 units
  int4* desc;       // [kMaxCtas]: the split item that CTA c begins: {rows, first token, kv head, last CTA}; rows 0: none
};

__device__ int g_paged_status;

// One sequence's queries and keys.
struct Seq {
  int c0, n;        // query tokens [c0, c0 + n)
  int ctx, kv_len;  // keys before them, and in all (0: no keys, or lengths that do not fit)
};

__device__ __forceinline__ Seq seq_at(const Params& p, int b, bool& bad) {
  Seq s{0, 0, 0, 0};
  if (b >= p.rows) return s;
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), len = __ldg(p.lens + b);
  if (c0 < 0 || c1 < c0 || c1 > p.n_tokens) {
    bad = true;
    return s;
  }
  s.c0 = c0;
  s.n = c1 - c0;
  if (s.n == 0) return s;
  if (len < s.n || len > p.max_pages * p.page_size) {
    bad = true;
    return s;
  }
  s.ctx = len - s.n;
  s.kv_len = len;
  return s;
}

// The key tiles that row tile rt of a sequence visits: the first n_sink, then from j0 on.
struct Tiles {
  int steps, n_sink, j0;
};

__device__ __forceinline__ Tiles tiles_of(const Params& p, const Seq& s, int rt) {
  Tiles t{1, 0, 0};  // a sequence without keys visits one tile, all of it masked
  if (s.kv_len == 0) return t;
  const int first = rt * p.R;
  const int hi = p.mask ? s.kv_len : s.ctx + min(first + p.R, s.n);
  const int n_hi = (hi + BN - 1) / BN;
  if (p.window > 0) {
    // no row's window begins earlier (a drafted token that sees none is at ctx - 1)
    const int lo = max((p.mask ? s.ctx - 1 : s.ctx + first) - p.window + 1, 0);
    t.j0 = min(lo / BN, n_hi - 1);
    t.n_sink = min((min(p.sinks, hi) + BN - 1) / BN, t.j0);
  }
  t.steps = t.n_sink + n_hi - t.j0;
  return t;
}

// What a CTA does of one (row tile, kv head): steps [s0, s1) of its tiles.
struct Item {
  int tok0;         // first query token (into q)
  int first, ntok;  // ... its place among the sequence's newest tokens; tokens of the item
  int h;            // kv head
  int s0, s1;
  int n_sink, j0;
  int ctx, kv_len;
  int seq_n;  // the sequence's newest tokens
  int out;    // where the result goes: 0 O and LSE, 1 the CTA's first partial, 2 its second
  __device__ __forceinline__ int tile(int s) const { return s < n_sink ? s : j0 + s - n_sink; }
};
constexpr int kItemWords = 12;
static_assert(sizeof(Item) == 4 * kItemWords, "published word by word");

__device__ __forceinline__ uint8_t* align_1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint64_t timeout_ns) {
  const bool ok = mbar_wait_bounded(bar, parity, abort_flag, timeout_ns);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void record_abort(volatile uint32_t* abort_flag, int site) {
  *abort_flag = 1;
  atomicCAS(&g_paged_status, 0, site);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Bits [lo, hi) of a 32-bit word whose first bit stands for `base`.
__device__ __forceinline__ uint32_t range_bits(int base, int lo, int hi) {
  const int a = max(lo - base, 0), b = min(hi - base, 32);
  if (a >= b) return 0u;
  return (0xFFFFFFFFu >> (32 - (b - a))) << a;
}

// A NaN in either half of a pair of fp16?
__device__ __forceinline__ bool has_nan_f16x2(uint32_t w) {
  return (w & 0x7FFFu) > 0x7C00u || ((w >> 16) & 0x7FFFu) > 0x7C00u;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Params p) {
  using C = Cfg<D>;
  constexpr int KS = C::kK, VS = C::kV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  uint8_t* q_s = smem;                      // two Q buffers
  uint8_t* k_s = smem + 2 * C::kTileBytes;
  uint8_t* v_s = k_s + KS * C::kTileBytes;
  __shared__ uint64_t k_full[KS], k_empty[KS], v_full[VS], v_empty[VS];
  __shared__ uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done, o_full, o_empty, mma_drain;
  __shared__ uint64_t seq_full[kSeqSlots], seq_empty[kSeqSlots];
  __shared__ int item_words[kSeqSlots][kItemWords];
  // Step g's V tile has been converted, and which of its keys hold a NaN, at g % kReady.  A softmax
  // warp looks at them after handing over P(g), when the conversion may be up to VS steps ahead;
  // with more places than that neither is reused under it.
  constexpr int kReady = 8;
  static_assert(VS < kReady, "read before it is used again");
  __shared__ uint64_t v_ready[kReady];
  __shared__ __align__(16) uint32_t nan_keys[kReady][4];
  __shared__ uint32_t tmem_base_slot, abort_flag;

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  griddep_launch_dependents();

  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < kReady; ++s) mbar_init(&v_ready[s], 4);  // one arrival per converting warp
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 2);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    mbar_init(&pv_done, 1);
    mbar_init(&o_full, 1);
    mbar_init(&o_empty, 128);
    mbar_init(&mma_drain, 1);
    for (int i = 0; i < kSeqSlots; ++i) {
      mbar_init(&seq_full[i], 1);
      mbar_init(&seq_empty[i], kSeqConsumers);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_slot;
  volatile uint32_t* abort_v = &abort_flag;
  // the CTA's k-th item (s1 == 0: no more); false when a wait gave up
  auto next_item = [&](int k, Item& it) {
    if (!warp_wait(&seq_full[k % kSeqSlots], (k / kSeqSlots) & 1, abort_v, kTimeoutNs)) return false;
    volatile int* w = item_words[k % kSeqSlots];
    int* dst = reinterpret_cast<int*>(&it);
#pragma unroll
    for (int i = 0; i < kItemWords; ++i) dst[i] = w[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seq_empty[k % kSeqSlots]);
    return true;
  };

  if (warp >= 8) {
    regs_decrease<kRegsOther>();
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------ plan, then TMA producer
      if (lane == 0) {
        tma_prefetch_map(&tk);
        tma_prefetch_map(&tv);
      }
      bool bad = false;
      // key tiles of sequence b, over its row tiles and kv heads
      auto weight = [&](int b) {
        const Seq s = seq_at(p, b, bad);
        int64_t w = 0;
        for (int rt = 0; rt * p.R < s.n; ++rt) w += tiles_of(p, s, rt).steps;
        return w * p.Hkv;
      };
      const int64_t w_first = weight(lane);  // the first 32 sequences' stay in registers
      int64_t total = w_first;
      for (int b = 32 + lane; b < p.rows; b += 32) total += weight(b);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
      const int64_t per = (total + gridDim.x - 1) / gridDim.x;
      int64_t at = per * blockIdx.x;  // this CTA's part of the list: [at, end)
      const int64_t end = min(at + per, total);
      int b = 0, rt = 0, h = 0, s0 = 0;
      Seq seq{0, 0, 0, 0};
      Tiles t{1, 0, 0};
      if (at < end) {
        // the sequence that holds `at`, then the row tile, the kv head and the step
        int64_t before = 0;
        for (int base = 0; base < p.rows; base += 32) {
          const int64_t w = base == 0 ? w_first : weight(base + lane);
          int64_t incl = w;
#pragma unroll
          for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, before + incl > at);
          if (past) {
            const int l = __ffs(past) - 1;
            b = base + l;
            before += __shfl_sync(0xffffffffu, incl - w, l);
            break;
          }
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
        seq = seq_at(p, b, bad);
        int64_t rem = at - before;
        for (; rt * p.R < seq.n; ++rt) {
          t = tiles_of(p, seq, rt);
          const int64_t here = static_cast<int64_t>(t.steps) * p.Hkv;
          if (rem < here) break;
          rem -= here;
        }
        h = static_cast<int>(rem / t.steps);
        s0 = static_cast<int>(rem % t.steps);
        if (rt * p.R >= seq.n || h >= p.Hkv) at = end;  // the lengths changed under the call
      }
      if (bad) atomicCAS(&g_paged_status, 0, kSiteInput);
      int4 desc = make_int4(0, 0, 0, 0);
      uint32_t g = 0, v_loads = 0;  // steps whose K, and whose V, is on its way
      bool ok = true;
      const int per_tile = p.page_size >= BN ? 1 : BN / p.page_size;  // pages of a tile
      const int box_rows = min(p.page_size, BN);
      for (int k = 0; ok; ++k) {
        Item item;
        const bool more = at < end;
        item.s0 = s0;
        item.s1 = more ? static_cast<int>(min(static_cast<int64_t>(t.steps), s0 + (end - at))) : 0;
        item.first = rt * p.R;
        item.ntok = min(p.R, seq.n - item.first);
        item.tok0 = seq.c0 + item.first;
        item.h = h;
        item.n_sink = t.n_sink;
        item.j0 = t.j0;
        item.ctx = seq.ctx;
        item.kv_len = seq.kv_len;
        item.seq_n = seq.n;
        item.out = item.s0 == 0 && item.s1 == t.steps ? 0 : item.s0 == 0 ? 2 : 1;
        if (k >= kSeqSlots) ok = warp_wait(&seq_empty[k % kSeqSlots], (k / kSeqSlots - 1) & 1, abort_v, kTimeoutNs);
        if (!ok) break;
        if (lane == 0) {
          const int* src = reinterpret_cast<const int*>(&item);
#pragma unroll
          for (int i = 0; i < kItemWords; ++i) item_words[k % kSeqSlots][i] = src[i];
          mbar_arrive(&seq_full[k % kSeqSlots]);
        }
        __syncwarp();
        if (!more) break;
        if (item.out == 2) {  // the CTAs after this one hold the rest of the item
          const int64_t last = at - s0 + t.steps - 1;
          desc = make_int4(item.ntok * p.G, item.tok0, h, static_cast<int>(last / per));
        }
        // pages [win, win + 32) of the row, one per lane, and the next 32 on their way
        const int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages;
        const int used = (item.kv_len + p.page_size - 1) / p.page_size;
        auto load_ids = [&](int w) { return w + lane < used ? __ldg(row + w + lane) : 0; };
        int win = -64, ids = 0, ids_next = 0;
        for (int s = item.s0; s < item.s1 && ok; ++s) {
          const int key0 = item.tile(s) * BN;
          const int page0 = key0 / p.page_size, slot0 = key0 % p.page_size;
          if (page0 / 32 * 32 != win) {
            const int w = page0 / 32 * 32;
            ids = w == win + 32 ? ids_next : load_ids(w);
            ids_next = load_ids(w + 32);
            win = w;
          }
          // lane page0 - win + i loads the tile's page i, if the sequence reaches it
          const int i = lane - (page0 - win);
          const bool mine = i >= 0 && i < per_tile && key0 + i * box_rows < item.kv_len;
          int page = ids;
          if (mine && (page < 0 || page >= p.n_pages)) {
            atomicCAS(&g_paged_status, 0, kSiteInput);
            page = max(p.n_pages, 1);  // past the pool: reads as zeros
          }
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * static_cast<uint32_t>(box_rows * D * 2);
          // the page's slots into ring slot `slot` of K or V
          auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full) {
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            if (mine) {
#pragma unroll
              for (int cb = 0; cb < D / 64; ++cb)
                tma_load_4d(dst + cb * C::kColBlockBytes + i * box_rows * 128, map, full, cb * 64, slot0, h, page);
            }
            __syncwarp();
          };
          if (g >= KS) ok = warp_wait(&k_empty[g % KS], (g / KS - 1) & 1, abort_v, kTimeoutNs);
          if (!ok) break;
          load(&tk, k_s + (g % KS) * C::kTileBytes, &k_full[g % KS]);
          ++g;
          if (v_loads >= VS) ok = warp_wait(&v_empty[v_loads % VS], (v_loads / VS - 1) & 1, abort_v, kTimeoutNs);
          if (!ok) break;
          load(&tv, v_s + (v_loads % VS) * C::kTileBytes, &v_full[v_loads % VS]);
          ++v_loads;
        }
        // the next (row tile, kv head)
        at += item.s1 - item.s0;
        s0 = 0;
        if (at < end && ++h == p.Hkv) {
          h = 0;
          ++rt;
          if (rt * p.R >= seq.n) {
            rt = 0;
            do {
              seq = seq_at(p, ++b, bad);
            } while (seq.n == 0 && b < p.rows);
          }
          t = tiles_of(p, seq, rt);
        }
      }
      if (!ok) {
        if (lane == 0) record_abort(abort_v, kSiteProducer);
        desc = make_int4(0, 0, 0, 0);
        // unwinding: let the copies in flight land before the CTA exits
        for (uint32_t i = (g > KS ? g - KS : 0); i < g; ++i)
          mbar_wait_bounded(&k_full[i % KS], (i / KS) & 1, abort_v, kDrainTimeoutNs);
        for (uint32_t i = (v_loads > VS ? v_loads - VS : 0); i < v_loads; ++i)
          mbar_wait_bounded(&v_full[i % VS], (i / VS) & 1, abort_v, kDrainTimeoutNs);
      }
      if (lane == 0) p.desc[blockIdx.x] = desc;
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ tcgen05 issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(BM, D, true);
      const uint32_t q_addr = smem_u32(q_s), k_addr = smem_u32(k_s), v_addr = smem_u32(v_s);
      static_assert(C::kColBlockBytes == 16384, "K-step offsets of mma_bf16_ss_k8");
      // S of step g from Q buffer qb
      auto issue_s = [&](uint32_t g, uint32_t qb) {
        const uint32_t slot = g % KS;
        const uint64_t qd = sdesc_sw128(opaque(q_addr) + qb * C::kTileBytes, 16, 1024);
        const uint64_t kd = sdesc_sw128(opaque(k_addr) + slot * C::kTileBytes, 16, 1024);
        if constexpr (D == 128)
          mma_bf16_ss_k8(tmem + (g & 1) * BN, qd, kd, idesc_s, smem_u32(&s_full[g & 1]), smem_u32(&k_empty[slot]));
        else
          mma_bf16_ss_k4(tmem + (g & 1) * BN, qd, kd, idesc_s, smem_u32(&s_full[g & 1]), smem_u32(&k_empty[slot]));
      };
      auto issue_pv = [&](uint32_t g, bool accumulate) {
        const uint32_t slot = g % VS;
        const uint64_t vd = sdesc_sw128(opaque(v_addr) + slot * C::kTileBytes, C::kColBlockBytes, 1024);
        mma_bf16_ts_k8(tmem + kTmemO, tmem + (g & 1) * BN + 64, vd, idesc_pv, accumulate ? 1u : 0u,
                       smem_u32(&pv_done), smem_u32(&v_empty[slot]));
      };
      auto wait_k = [&](uint32_t n) { return warp_wait(&k_full[n % KS], (n / KS) & 1, abort_v, kTimeoutNs); };
      // first S of item k (steps from g on)
      auto begin = [&](int k, uint32_t g) {
        if (!warp_wait(&q_full[k & 1], (k >> 1) & 1, abort_v, kTimeoutNs) || !wait_k(g)) return false;
        tc_fence_after();
        issue_s(g, k & 1);
        return true;
      };
      uint32_t g = 0;
      Item item;
      bool ok = next_item(0, item);
      if (ok && item.s1 > 0) {
        ok = begin(0, 0);
        if (ok && item.s1 - item.s0 == 1) mma_commit_elect(&q_empty[0]);
      }
      for (int k = 0; ok && item.s1 > 0; ++k) {
        const int n = item.s1 - item.s0;
        Item next;
        next.s0 = next.s1 = 0;
        for (int j = 0; j < n && ok; ++j, ++g) {
          // S of the next step: this item's, or the next item's first
          if (j + 1 < n) {
            ok = wait_k(g + 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(g + 1, k & 1);
            if (j + 2 == n) mma_commit_elect(&q_empty[k & 1]);  // the item's last S has been issued
          } else {
            ok = next_item(k + 1, next);
            if (ok && next.s1 > 0) {
              ok = begin(k + 1, g + 1);
              if (ok && next.s1 - next.s0 == 1) mma_commit_elect(&q_empty[(k + 1) & 1]);
            }
            if (!ok) break;
          }
          ok = warp_wait(&v_ready[g % kReady], (g / kReady) & 1, abort_v, kTimeoutNs);
          if (ok && j == 0 && k > 0) ok = warp_wait(&o_empty, (k - 1) & 1, abort_v, kTimeoutNs);
          if (ok) ok = warp_wait(&p_full[g & 1], (g >> 1) & 1, abort_v, kTimeoutNs);
          if (!ok) break;
          tc_fence_after();
          issue_pv(g, j > 0);
          if (j + 1 == n) mma_commit_elect(&o_full);  // the item's O is complete
        }
        item = next;
      }
      if (!ok && lane == 0) record_abort(abort_v, kSiteIssuer);
      mma_commit_elect(&mma_drain);
      warp_wait(&mma_drain, 0, abort_v, ok ? kTimeoutNs : kDrainTimeoutNs);
    } else {
      // ------------------------------------------------------------ Q rows
      // Row r = token * G + head of the group, stored as a 128-byte-swizzled K-major tile; rows
      // past the item's keep what the buffer held (their S rows are not used).
      constexpr int kChunks = D / 8, kUnroll = 8;
      const int me = (warp - 10) * 32 + lane;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        Item item;
        ok = next_item(k, item);
        if (!ok || item.s1 == 0) break;
        if (k >= 2) ok = warp_wait(&q_empty[k & 1], (k / 2 - 1) & 1, abort_v, kTimeoutNs);
        if (!ok) break;
        uint8_t* dst = q_s + (k & 1) * C::kTileBytes;
        const int pieces = item.ntok * p.G * kChunks;
        for (int e0 = me; e0 < pieces; e0 += 64 * kUnroll) {
          uint4 x[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int e = e0 + 64 * u, r = e / kChunks, ch = e % kChunks;
            if (e < pieces)
              x[u] = __ldg(reinterpret_cast<const uint4*>(p.q + (item.tok0 + r / p.G) * p.q_token +
                                                          (item.h * p.G + r % p.G) * p.q_head + ch * 8));
          }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int e = e0 + 64 * u, r = e / kChunks, ch = e % kChunks;
            if (e < pieces)
              *reinterpret_cast<uint4*>(dst + (ch / 8) * C::kColBlockBytes + r * 128 +
                                        (((ch % 8) ^ (r & 7)) << 4)) = x[u];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[k & 1]);
      }
      if (!ok && lane == 0) record_abort(abort_v, kSiteQuery);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ V to fp16
    // Warp w takes rows 32 w .. 32 w + 31 of each V tile; a lane's 16-byte chunk holds
    // 8 values of one row.  Rows past the sequence become 0, whatever the page holds. A NaN
    // becomes 0 too and is noted for its key: the rows that see the key get NaN in
    // the epilogue, a row that does not is not reached through 0 * NaN.
    regs_decrease<kRegsConvert>();
    constexpr int kBlocks = D / 64, kPieces = 8 * kBlocks;  // 16-byte chunks per lane
    const int w = warp - 4;
    uint32_t g = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item item;
      ok = next_item(k, item);
      if (!ok || item.s1 == 0) break;
      for (int s = item.s0; s < item.s1; ++s, ++g) {
        const uint32_t slot = g % VS;
        ok = warp_wait(&v_full[slot], (g / VS) & 1, abort_v, kTimeoutNs);
        if (!ok) break;
        const int valid = item.kv_len - item.tile(s) * BN;  // rows of the tile that are tokens
        const uint32_t base = smem_u32(v_s + slot * C::kTileBytes) + w * 32 * 128 + lane * 16;
        uint4 x[kPieces];
        uint32_t nans = 0;  // a bit per chunk
#pragma unroll
        for (int u = 0; u < kPieces; ++u) x[u] = lds128(base + (u / 8) * C::kColBlockBytes + (u % 8) * 512);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          const int r = 32 * w + 4 * (u % 8) + lane / 8;
          const bool live = r < valid;
          x[u].x = live ? bf16x2_to_f16x2(x[u].x) : 0u;
          x[u].y = live ? bf16x2_to_f16x2(x[u].y) : 0u;
          x[u].z = live ? bf16x2_to_f16x2(x[u].z) : 0u;
          x[u].w = live ? bf16x2_to_f16x2(x[u].w) : 0u;
          if (has_nan_f16x2(x[u].x) || has_nan_f16x2(x[u].y) || has_nan_f16x2(x[u].z) || has_nan_f16x2(x[u].w))
            nans |= 1u << u;
        }
        uint32_t keys = 0;
        if (__any_sync(0xffffffffu, nans != 0)) {
#pragma unroll
          for (int u = 0; u < kPieces; ++u) {
            uint32_t* y = reinterpret_cast<uint32_t*>(&x[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if ((y[i] & 0x7FFFu) > 0x7C00u) y[i] &= 0xFFFF0000u;
              if (((y[i] >> 16) & 0x7FFFu) > 0x7C00u) y[i] &= 0x0000FFFFu;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, (nans >> u) & 1u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((hit >> (8 * i)) & 0xFFu) keys |= 1u << (4 * (u % 8) + i);
          }
        }
#pragma unroll
        for (int u = 0; u < kPieces; ++u) sts128(base + (u / 8) * C::kColBlockBytes + (u % 8) * 512, x[u]);
        if (lane == 0) nan_keys[g % kReady][w] = keys;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ready[g % kReady]);
      }
    }
    if (!ok && lane == 0) record_abort(abort_v, kSiteConvert);
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    regs_increase<kRegsSoftmax>();
    const int r_in = warp * 32 + lane;  // row of the item
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + kTmemO;
    const float c = p.c;
    uint32_t g = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item item;
      ok = next_item(k, item);
      if (!ok || item.s1 == 0) break;
      const int rows = item.ntok * p.G;
      const bool live = r_in < rows;
      const bool warp_live = warp * 32 < rows;
      const int u_tok = r_in / p.G;       // token of the row within the item
      const int u = item.first + u_tok;   // ... among the sequence's newest tokens
      const uint32_t* words = (p.mask && live) ? p.mask + static_cast<int64_t>(item.tok0 + u_tok) * p.mask_words : nullptr;
      const int n_words = min(p.mask_words, (item.seq_n + 31) / 32);
      // the row's limits: keys [lo, hi) and the sinks below hi; drafted tokens by the mask
      const int hi = !live || item.kv_len == 0 ? 0 : p.mask ? item.ctx : item.ctx + u + 1;
      int lo = 0;
      if (p.window > 0) {
        int place = item.ctx + u;
        if (words) {
          place = item.ctx - 1;
          for (int i = 0; i < n_words; ++i) place += __popc(__ldg(words + i) & range_bits(32 * i, 0, item.seq_n));
        }
        lo = place - p.window + 1;
      }
      const int sinks = p.window > 0 ? p.sinks : 0;
      // tiles that every row of the item sees whole: below `whole_hi` and from `whole_lo` on
      const int whole_hi = item.kv_len == 0 ? 0 : p.mask ? item.ctx : item.ctx + item.first + 1;
      const int whole_lo = p.window > 0 ? item.ctx + (p.mask ? item.seq_n : item.first + item.ntok) - p.window : 0;
      float m = -INFINITY;   // reference value, log2 units
      float l = 0.0f;        // sum of the fp16-rounded P (normalises O)
      float l_exact = 0.0f;  // sum of the fp32 P (gives LSE)
      bool nan_row = false;
      for (int s = item.s0; s < item.s1; ++s, ++g) {
        const int key0 = item.tile(s) * BN;
        const bool masked = key0 + BN > whole_hi || (key0 < whole_lo && key0 + BN > sinks);
        uint32_t vis[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
        if (masked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 32 * i;
            vis[i] = range_bits(key, lo, hi) | range_bits(key, 0, min(sinks, hi));
            if (words) {
              const int u0 = key - item.ctx;  // the drafted token of the word's first bit
              const int at = u0 >> 5;
              const uint32_t a = at >= 0 && at < n_words ? __ldg(words + at) : 0u;
              const uint32_t z = at + 1 >= 0 && at + 1 < n_words ? __ldg(words + at + 1) : 0u;
              if (item.kv_len > 0) vis[i] |= __funnelshift_r(a, z, u0 & 31) & range_bits(u0, 0, item.seq_n);
            }
          }
        } else if (!live) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vis[i] = 0u;
        }
        ok = warp_wait(&s_full[g & 1], (g >> 1) & 1, abort_v, kTimeoutNs);
        if (!ok) break;
        if (!warp_live) {  // no row: nothing of these lanes is ever read
          mbar_arrive(&p_full[g & 1]);
          continue;
        }
        tc_fence_after();
        const uint32_t s_tmem = tmem + lane_off + (g & 1) * BN;
        uint32_t r[128];
        tmem_ld128_wait(s_tmem, r);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 128; ++i) r[i] = (vis[i / 32] >> (i % 32)) & 1u ? r[i] : __float_as_uint(-INFINITY);
        }
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 128; i += 8) {
          mx0 = max3f(mx0, __uint_as_float(r[i + 0]), __uint_as_float(r[i + 1]));
          mx1 = max3f(mx1, __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
          mx2 = max3f(mx2, __uint_as_float(r[i + 4]), __uint_as_float(r[i + 5]));
          mx3 = max3f(mx3, __uint_as_float(r[i + 6]), __uint_as_float(r[i + 7]));
        }
        const float top = live ? fmaxf(max3f(mx0, mx1, mx2), mx3) * c : -INFINITY;
        // m moves when the row sees its first key, or P would pass 2^15
        float alpha = 1.0f;
        if (top > m + kLimit || (m == -INFINITY && top > -INFINITY)) {
          const float m_new = top - kStart;
          alpha = ex2_approx(m - m_new);  // 0 from -inf
          m = m_new;
          l *= alpha;
          l_exact *= alpha;
        }
        if (s > item.s0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          // PV(g-1) has to be complete.  PV(g-2) is, as S(g) was issued after it, and PV(g) waits for
          // this warp, so the barrier is in phase g-1 or has just left it
          ok = warp_wait(&pv_done, (g - 1) & 1, abort_v, kTimeoutNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t o[32];
            tmem_ld32_wait(o_tmem + cb * 32, o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0, x1;
              f2_unpack(fmul2(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), x0, x1);
              o[i] = __float_as_uint(x0);
              o[i + 1] = __float_as_uint(x1);
            }
            tmem_st32(o_tmem + cb * 32, o);
          }
        }
        const float neg_m = m == -INFINITY ? 0.0f : -m;
        const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(neg_m, neg_m);
        uint64_t e0 = f2_pack(0.0f, 0.0f), e1 = e0;
        float q0 = 0.0f, q1 = 0.0f, q2 = 0.0f, q3 = 0.0f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int e = 64 * half + 2 * i;
            float x0, x1;
            f2_unpack(ffma2(f2_pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2, nm2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            pk[i] = pack_f16x2(p0, p1);
            if (i & 1) {
              e1 = fadd2(e1, f2_pack(p0, p1));
              add_f16x2_to_f32(q2, q3, pk[i]);
            } else {
              e0 = fadd2(e0, f2_pack(p0, p1));
              add_f16x2_to_f32(q0, q1, pk[i]);
            }
          }
          tmem_st32(s_tmem + 64 + 32 * half, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[g & 1]);
        float a0, a1, b0, b1;
        f2_unpack(e0, a0, a1);
        f2_unpack(e1, b0, b1);
        l_exact += (a0 + a1) + (b0 + b1);
        l += (q0 + q1) + (q2 + q3);
        // NaN among the V that the row sees
        ok = warp_wait(&v_ready[g % kReady], (g / kReady) & 1, abort_v, kTimeoutNs);
        if (!ok) break;
        const uint4 nk = lds128(smem_u32(nan_keys[g % kReady]));
        nan_row |= ((nk.x & vis[0]) | (nk.y & vis[1]) | (nk.z & vis[2]) | (nk.w & vis[3])) != 0;
      }
      if (!ok) break;
      // ---- epilogue, when the item's last PV is complete
      ok = warp_wait(&o_full, k & 1, abort_v, kTimeoutNs);
      if (!ok) break;
      tc_fence_after();
      // l is NaN when S or P was; a row without keys has l == 0
      const bool none = l == 0.0f && !nan_row;
      const float inv = none ? 0.0f : nan_row ? __int_as_float(0x7FC00000) : 1.0f / l;
      const float lse2 = none ? -INFINITY : m + lg2_approx(l_exact);
      const bool whole = item.out == 0;
      const int64_t at = whole ? static_cast<int64_t>(item.tok0 + u_tok) * p.Hq + item.h * p.G + r_in % p.G
                               : static_cast<int64_t>(2 * blockIdx.x + item.out - 1) * BM + r_in;
      if (warp_live) {
        // 32 columns at a time; O of a row without keys is whatever the MMA made of P = 0, and not used
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          tmem_ld32_wait(o_tmem + 32 * cb, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
          if (live && whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + 32 * cb);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__uint_as_float(o[8 * ch + 2 * i]), __uint_as_float(o[8 * ch + 2 * i + 1]));
              dst[ch] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (live) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * D + 32 * cb);
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              dst[ch] = make_uint4(o[4 * ch], o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]);
          }
        }
        if (live) {
          if (whole)
            p.lse[at] = lse2 * 0.69314718055994531f;
          else
            p.part_lse[at] = lse2;
        }
      }
      tc_fence_before();
      mbar_arrive(&o_empty);  // the next item's first PV may overwrite O
    }
    if (!ok && lane == 0) record_abort(abort_v, kSiteSoftmax);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The item that CTA blockIdx.x began and left to the CTAs after it: O and LSE of its partials,
//     LSE = log2 sum_r 2^LSE_r,   O = sum_r 2^(LSE_r - LSE) O_r,
// one warp per row, the ranges in order.  A range that sees no key (LSE_r = -inf) has weight 0.
template <int D>
__global__ void __launch_bounds__(256) attn_tree_merge_kernel(const Params p) {
  constexpr int kVec = D / 32;
  griddep_wait();
  const int4 d = p.desc[blockIdx.x];
  const int lane = threadIdx.x % 32;
  const int row = blockIdx.y * 8 + threadIdx.x / 32;
  if (row >= d.x) return;
  const int n = d.w - static_cast<int>(blockIdx.x) + 1;  // ranges: slot 1 of this CTA, slot 0 of the next ones
  auto slot = [&](int i) { return static_cast<int64_t>(2 * (blockIdx.x + i) + (i == 0)) * BM + row; };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, p.part_lse[slot(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float ref = top == -INFINITY ? 0.0f : top;
  float acc[kVec] = {}, sum = 0.0f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float w = ex2_approx(p.part_lse[slot(i)] - ref);
    const float* src = p.part_o + slot(i) * D + lane * kVec;
    sum += w;
#pragma unroll
    for (int v = 0; v < kVec; v += 2) {
      const float2 x = *reinterpret_cast<const float2*>(src + v);
      acc[v] += w * x.x;
      acc[v + 1] += w * x.y;
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = static_cast<int64_t>(d.y + row / p.G) * p.Hq + d.z * p.G + row % p.G;
#pragma unroll
  for (int v = 0; v < kVec; v += 2)
    *reinterpret_cast<uint32_t*>(p.o + at * D + lane * kVec + v) = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
  if (lane == 0) p.lse[at] = sum == 0.0f ? -INFINITY : (ref + lg2_approx(sum)) * 0.69314718055994531f;
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
thread_local cudaError_t t_last_cuda_error = cudaSuccess;

int cuda_fail(cudaError_t e) {
  t_last_cuda_error = e;
  return ATTN_ERR_CUDA;
}

// Kernel attributes, once per device.
int prepare_device(int dev) {
  constexpr int kMax = 64;
  static std::mutex mutex;
  static bool ready[kMax];
  if (dev < 0 || dev >= kMax) return ATTN_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(mutex);
  if (ready[dev]) return ATTN_OK;
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(attn_tree_kernel<128>),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<128>::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(attn_tree_kernel<64>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<64>::kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e);
  if (!attn_host::encode_tiled_fn()) return ATTN_ERR_TENSOR_MAP;
  ready[dev] = true;
  return ATTN_OK;
}

// Pages as [page][head][slot][D] with any strides, read in boxes of 64 columns x up to 128
// slots of one head and page.  A pool without pages reads as zeros everywhere: its map
// covers one page at `some` (never read: every page number is past it).
bool encode_pages(CUtensorMap* map, const attn_kv_cache& c, const void* base, int64_t page, int64_t head, int64_t slot,
                  const void* some) {
  attn_host::EncodeTiledFn fn = attn_host::encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(std::max(c.n_pages, 1))};
  // the stride of a dimension of one element is not used, but has to be valid
  auto bytes = [&](int64_t stride, int64_t size) {
    return static_cast<cuuint64_t>(size > 1 && c.n_pages > 0 ? stride * 2 : c.D * 2);
  };
  const cuuint64_t strides[3] = {bytes(slot, c.page_size), bytes(head, c.Hkv), bytes(page, c.n_pages)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(std::min(c.page_size, BN)), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(c.n_pages > 0 ? base : some), dims, strides, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Workspace {
  size_t o, lse, desc, bytes;  // offsets, and in all
};

Workspace layout(int D) {
  Workspace w;
  w.o = 0;
  w.lse = w.o + sizeof(float) * kMaxCtas * 2 * BM * D;
  w.desc = w.lse + sizeof(float) * kMaxCtas * 2 * BM;
  w.bytes = w.desc + sizeof(int4) * kMaxCtas;
  return w;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

template <int D>
int launch(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int sms, cudaStream_t stream) {
  const int grid = std::min(sms, kMaxCtas);
  attn_tree_kernel<D><<<grid, kThreads, Cfg<D>::kSmemBytes, stream>>>(tk, tv, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (std::min(p.R, p.n_tokens) * p.G + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<D>, p);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

size_t attn_fwd_tree_workspace_size(int D) { return D == 64 || D == 128 ? layout(D).bytes : 0; }

int attn_fwd_tree(const attn_kv_cache* cache, const void* q, int64_t q_stride_token, int64_t q_stride_head, void* o,
                  float* lse, int n_tokens, int Hq, const int32_t* cu_tokens, const uint32_t* tree_mask,
                  int mask_words, int window, int sinks, float scale, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  // ---- argument checks (host only, before any CUDA call)
  int st = attn_host::check_cache(cache, true, false);
  if (st != ATTN_OK) return st;
  const attn_kv_cache& c = *cache;
  if (n_tokens < 0 || Hq < 1 || Hq % c.Hkv != 0 || Hq / c.Hkv > BM) return ATTN_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || !(std::isfinite(scale) && scale > 0.0f)) return ATTN_ERR_INVALID_ARG;
  if (tree_mask ? mask_words < 1 : mask_words != 0) return ATTN_ERR_INVALID_ARG;
  if (q_stride_token < 0 || q_stride_head < 0 || q_stride_token % 8 != 0 || q_stride_head % 8 != 0)
    return ATTN_ERR_INVALID_ARG;
  if (n_tokens == 0 || c.rows == 0) return ATTN_OK;
  if (!q || !o || !lse || !cu_tokens || !workspace) return ATTN_ERR_NULL_PTR;
  const void* wide[] = {q, o, lse, workspace};
  for (const void* ptr : wide)
    if (!attn_host::aligned_to(ptr, 16)) return ATTN_ERR_MISALIGNED;
  if (!attn_host::aligned_to(cu_tokens, 4) || !attn_host::aligned_to(tree_mask, 4)) return ATTN_ERR_MISALIGNED;
  const Workspace w = layout(c.D);
  if (workspace_bytes < w.bytes) return ATTN_ERR_INVALID_ARG;
  const int64_t heads = static_cast<int64_t>(n_tokens) * Hq;
  const int64_t kv_end[] = {(c.n_pages - 1) * c.k_stride_page + (c.Hkv - 1) * c.k_stride_head +
                                (c.page_size - 1) * c.k_stride_slot + c.D,
                            (c.n_pages - 1) * c.v_stride_page + (c.Hkv - 1) * c.v_stride_head +
                                (c.page_size - 1) * c.v_stride_slot + c.D};
  const struct {
    const void* at;
    size_t bytes;
  } outs[] = {{o, static_cast<size_t>(heads) * c.D * 2}, {lse, static_cast<size_t>(heads) * 4}, {workspace, w.bytes}},
    ins[] = {{q, static_cast<size_t>((n_tokens - 1) * q_stride_token + (Hq - 1) * q_stride_head + c.D) * 2},
             {c.n_pages > 0 ? c.k : nullptr, static_cast<size_t>(std::max<int64_t>(kv_end[0], 0)) * 2},
             {c.n_pages > 0 ? c.v : nullptr, static_cast<size_t>(std::max<int64_t>(kv_end[1], 0)) * 2},
             {c.page_table, static_cast<size_t>(c.rows) * c.max_pages * 4},
             {c.seq_lens, static_cast<size_t>(c.rows) * 4},
             {cu_tokens, (static_cast<size_t>(c.rows) + 1) * 4},
             {tree_mask, static_cast<size_t>(n_tokens) * mask_words * 4}};
  for (int a = 0; a < 3; ++a) {
    for (const auto& in : ins)
      if (overlaps(outs[a].at, outs[a].bytes, in.at, in.bytes)) return ATTN_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (overlaps(outs[a].at, outs[a].bytes, outs[b].at, outs[b].bytes)) return ATTN_ERR_INVALID_ARG;
  }

  // ---- device
  cudaError_t e;
  int dev = 0;
  const int sms = attn_host::device_sms(&e, &dev);
  if (sms < 0) return cuda_fail(e);
  if (sms == 0) return ATTN_ERR_UNSUPPORTED_DEVICE;
  st = prepare_device(dev);
  if (st != ATTN_OK) return st;
  CUtensorMap tk, tv;
  if (!encode_pages(&tk, c, c.k, c.k_stride_page, c.k_stride_head, c.k_stride_slot, q) ||
      !encode_pages(&tv, c, c.v, c.v_stride_page, c.v_stride_head, c.v_stride_slot, q))
    return ATTN_ERR_TENSOR_MAP;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_token = q_stride_token;
  p.q_head = q_stride_head;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.cu = cu_tokens;
  p.lens = c.seq_lens;
  p.table = c.page_table;
  p.mask = tree_mask;
  p.mask_words = mask_words;
  p.rows = c.rows;
  p.max_pages = c.max_pages;
  p.n_pages = c.n_pages;
  p.page_size = c.page_size;
  p.n_tokens = n_tokens;
  p.Hq = Hq;
  p.Hkv = c.Hkv;
  p.G = Hq / c.Hkv;
  p.R = BM / p.G;
  p.window = std::min(window, 1 << 30);  // no key is further away (rows hold less than 2^31 tokens)
  p.sinks = std::min(sinks, 1 << 30);
  p.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.part_lse = reinterpret_cast<float*>(ws + w.lse);
  p.desc = reinterpret_cast<int4*>(ws + w.desc);
  return c.D == 128 ? launch<128>(tk, tv, p, sms, stream) : launch<64>(tk, tv, p, sms, stream);
}

const char* attn_paged_strerror(int status) { return attn_host::status_text(status, t_last_cuda_error); }

int attn_paged_debug_status(cudaStream_t stream, int* site) {
  if (site) *site = 0;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e);
  int value = 0;
  e = cudaMemcpyFromSymbol(&value, g_paged_status, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e);
  if (value != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  if (site) *site = value;
  return value == 0 ? ATTN_OK : value == kSiteInput ? ATTN_ERR_INVALID_ARG : ATTN_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
