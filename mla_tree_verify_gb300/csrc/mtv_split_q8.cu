// Split-K partial kernel of the e4m3 latent cache on the 5th-generation tensor cores
// (tcgen05 kind::f8f6f4 + TMEM).
//
// Mathematics.  Key column c holds codes x_c (576 e4m3 values) and a scale g_c; V is the first
// 512 codes.  With y_c = sm_scale log2(e) g_c <q, x_c> + log2 g_c the weight that multiplies
// codes is 2^{y_c}, so the kernel runs its online softmax over y, with a reference r for each
// column that trails the running maximum:
//   P_c = 2^{y_c - r},  O = sum_c P_c x_c[0:512],  l = sum_c P_c / g_c,
//   out = O / l,  lse = ln 2 (r + log2 l).
// r is set to the exact maximum less 7, and again when a score passes it by 12 (P <= 2^12): on a
// segment's first tile and seldom after, so that most tiles need no column maximum, no second
// barrier and no rescale of O.  (Less 8: bs 8, 1k-4k 78.5 us against 76.0, bs 1, 185k 380 against
// 374; less 6: 73.6 and 371, with the weights' full precision a binary order less deep.)
// A key whose latent codes are all zero (a row of zeros has scale 1, whatever the others') counts in l
// and adds nothing to O: any g_c would do for it, and where references are set it is taken as
// 2^-60, so that its own does not push the other keys' weights out of P's range.
// No value is dequantised: the codes go from HBM into the matrix instructions as they are.
// q and P have to be 8-bit operands too and are each the sum of two:
// - q (split_q_row, in the planner's launch): a row is scaled by a power of two to a largest
//   value in [128, 256) and taken as hi = e4m3(q), lo = e4m3(q - hi).  A bf16 value has 8
//   significant bits and e4m3 4, so hi + lo is q exactly down to 2^-9 of the row's largest
//   value, and within 2^-17 of that value below (half of e4m3's smallest step, 2^-9, to at
//   least 128); products and sums are fp32.  hi and lo are
//   stacked as 128 columns of one instruction, the width that the tensor cores need for their
//   full rate (64.7 clocks an instruction, as for 64 columns), so the exact scores cost no
//   more than rounded ones would.
// - P in [0, 2^12] as an e4m3 and an e5m2 value (split_weights).  Either may be the coarse part.
//   From 2^-6 up, 13 binary orders below a fresh reference's maximum and more below a later
//   one, the sum is off by at most 2^-8 of P (half a step of its finer part) and 2^-11 of the
//   f16 it starts from: what bf16 weights are off by.  Below, e4m3 nears its smallest step,
//   2^-9, and e5m2 keeps 3 bits down to 2^-14: rounded to nearest P would be off by up to an
//   eighth, alike for alike weights.  There lo is rounded up or down at random (a hash of the
//   key column; off by up to a quarter of P, to the right mean), so that the errors of many small
//   weights average out whatever they multiply.  (An offset that went by the row of the tile
//   kept the sum of the weights and lost values that repeat with position.)
//
// Layout on the SM.  One CTA per SM walks its share of (column group, key tile) units, as the
// 16-bit kernel does (plan, partial slots and merges are shared).  A key tile is 128 rows of
// 576 bytes: four chunks of [128 rows][128 latent dims] with the 128-byte swizzle and one of
// [128 rows][64 rope dims] with the 64-byte swizzle, 72 KB; two tile buffers fit beside the
// split q (72 KB), so the scores of tile j + 1 are computed while the softmax works on tile j.
// The 16-bit kernel has room for one tile and runs gather, scores, softmax and values in
// sequence.  Transposed products, key rows and value dims on the TMEM lanes:
//   S^T[128 keys][64 hi | 64 lo] = X . Q^T      (18 MMAs 128x128x32; two buffers)
//   O^T[512 dims][64 columns]   += X^T . P^T    (4 blocks x (e4m3, e5m2) x 4 MMAs 128x64x32)
// P^T hi (e4m3) goes over the tile's rope chunk, which the scores no longer need, lo into its own
// 8 KB.
//
// Warp roles: warps 0-3 gather rows (cp.async) and scales, warp 0 also loads q (TMA); one thread
// of warp 12 issues the scores and one of warp 13 the values, so that neither waits for the
// other's turn; warps 4-11 run the softmax, the rescale and the epilogue.
//
// Measured.  64 requests of 8k-64k keys, trees of 1 to 16 drafts: 2.52 ms, 1.01 PFLOP/s of
// attention arithmetic, 53% of the measured bf16 matrix peak; one request of 185k keys with 16
// drafts: 373 us, 58%.  A tile takes about 2.3 us (4400 clocks at 64 heads): its 50 MMAs 2750
// clocks when nothing is waited for, the softmax 1650-1850.  What bounds it is the cycle of one tile
// buffer, two tiles long: values 3000 clocks (the scores of the next tile share the tensor
// cores), the refill of the chunks released last 1800, their scores 600, the softmax, and about
// 600 of hand-offs.  A third buffer, which would take it off the path, does not fit beside q.
#include "mtv_split_common.cuh"
#include "mtv_q8.cuh"

namespace mtv {
namespace tq {

using namespace tc;

constexpr int kProducerWarps = 4;
constexpr int kSoftmaxWarps = 8;
constexpr int kScoreWarp = kProducerWarps + kSoftmaxWarps;      // 12
constexpr int kValueWarp = kScoreWarp + 1;                      // 13
constexpr int kThreads = 512;                                   // (warps 14, 15 are idle)
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kFirstSoftmaxThread = 32 * kProducerWarps;
// Registers: 512 threads launch with 128 each; the softmax's two warpgroups take 176 and the
// other two give 48 (2 x 128 x 80 + 256 x 176 = 512 x 128).
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= 512 * 128, "register split");
constexpr uint32_t kChunk = 128 * 128;      // [128 rows][128 dims]
constexpr uint32_t kRopeChunk = 128 * 64;   // [128 rows][64 dims]
constexpr uint32_t kTileBytes = 4 * kChunk + kRopeChunk;        // 73728
constexpr uint32_t kQOff = 0;               // rows 0-63 hi, 64-127 lo, laid out as a tile
constexpr uint32_t kKvOff = kTileBytes;
constexpr uint32_t kPLoOff = 3 * kTileBytes;
// The epilogue needs its scratch only when the values of its last tile are done and P^T lo is
// free: merge weights [16][64] or [64][8], slots [64], 1/l [64].
constexpr uint32_t kWOff = kPLoOff;
constexpr uint32_t kSlotOff = kWOff + kMergeGroup * 64 * 4;
constexpr uint32_t kInvLOff = kSlotOff + kNsplit * 4;
static_assert(kInvLOff + 64 * 4 <= kPLoOff + kRopeChunk, "epilogue scratch");
constexpr uint32_t kRedOff = kPLoOff + kRopeChunk;              // float [64][4]
constexpr uint32_t kRefOff = kRedOff + 64 * 4 * 4;              // float [64] minus the reference
constexpr uint32_t kFactorOff = kRefOff + 64 * 4;               // float [64] score factors
constexpr uint32_t kScaleOff = kFactorOff + 64 * 4;             // float [2][128] row scales
constexpr uint32_t kBarOff = kScaleOff + 2 * 128 * 4;
constexpr uint32_t kMiscOff = kBarOff + 272;                    // tmem slot, abort, ticket
constexpr uint32_t kSegOff = kMiscOff + 32;
constexpr uint32_t kSmemBytes = kSegOff + 48;
static_assert(kSmemBytes <= 232448, "dynamic shared memory of one CTA");
static_assert(sizeof(SegInfo) <= 48, "segment info block");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;             // S^T of tile buffer b at 256 + 128 b; O^T at 0..255
constexpr uint32_t kErrBadScale = 16u;
constexpr float kPBits = 7.f;               // P = 2^7 at a fresh reference's maximum
constexpr float kLag = 5.f;                 // how far (base 2) scores may rise above it
constexpr float kEmptyBits = 60.f, kEmptyInv = 0x1p60f;   // scale 2^-60 of a key without values
constexpr float kNoKey = -3e38f;            // reference of a column that has seen no key
constexpr uint32_t kHalfBar = 2;            // named barriers 2, 3: the four warps of a half

// Instruction descriptors of kind::f8f6f4 with e4m3 A and B, or for kIdescPV5 e5m2 B, and fp32 D.
constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kIdescQK = idesc_e4m3(128, 128, 0, 0);
constexpr uint32_t kIdescPV4 = idesc_e4m3(128, 64, 1, 1);
constexpr uint32_t kIdescPV5 = kIdescPV4 | (1u << 10);   // B is e5m2

// Shared-memory matrix descriptors (address and leading stride in the low word, 8-row stride,
// version and swizzle in the high word).  An MMA takes low words as a base and a constant
// offset and adds them itself: built as 64-bit values outside, descriptors were kept in
// registers or on the stack by the compiler, and an MMA took about 120 clocks to issue, twice
// what it takes to run.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return (saddr >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescSw128 = (1024 >> 4) | (1u << 14) | (2u << 29);   // 8 rows of 128 bytes
constexpr uint32_t kDescSw64 = (512 >> 4) | (1u << 14) | (4u << 29);     // 8 rows of 64 bytes

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint32_t a_lo, uint32_t a_off,
                                         uint32_t a_hi, uint32_t b_lo, uint32_t b_off,
                                         uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 a, b;\n setp.ne.b32 p, %8, 0;\n"
      " add.u32 x, %1, %2;\n add.u32 y, %4, %5;\n mov.b64 a, {x, %3};\n mov.b64 b, {y, %6};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %7, p;\n}\n"
      ::"r"(d_tmem), "r"(a_lo), "r"(a_off), "r"(a_hi), "r"(b_lo), "r"(b_off), "r"(b_hi), "r"(idesc),
        "r"(accumulate));
}
// 64B-swizzled offset of 16-byte granule g in row r of an [rows][64 B] chunk.
__device__ __forceinline__ uint32_t swz64(uint32_t r, uint32_t g) {
  return r * 64u + ((g ^ ((r >> 1) & 3u)) << 4);
}
// ptx::mbar_wait() for this kernel: the limit is kept by the SM clock (two clocks a nanosecond,
// the nearest whole number), whose reading is cheap, and the code is short: the roles' loops
// together outgrow the instruction caches (a fifth of the warps' time went into fetching).
template <bool kSpin>
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort,
                                        uint64_t limit_ns) {
  if (ptx::mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  do {
    if (kSpin ? ptx::mbar_test(bar, parity) : ptx::mbar_try(bar, parity)) return true;
  } while (!*abort && (uint64_t)(clock64() - t0) < 2 * limit_ns);
  return false;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint64_t limit_ns) {
  return wait_on<false>(bar, parity, abort, limit_ns);
}
// For a thread that issues MMAs: it polls, without the suspension that mbar_try allows.
__device__ __forceinline__ bool spin_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint64_t limit_ns) {
  return wait_on<true>(bar, parity, abort, limit_ns);
}

__device__ __forceinline__ const unsigned char* shfl_ptr(const unsigned char* v, int from) {
  return (const unsigned char*)__shfl_sync(0xffffffffu, (unsigned long long)v, from);
}
// Arrives once on `bar` when every cp.async that this thread issued so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_addr(bar)) : "memory");
}

struct Bars {
  uint64_t q_full, q_empty, p_full, pv_done, o_done, o_free;
  uint64_t s_full[2], s_free[2], sc_full[2], drain[2];
  uint64_t kv_full[2][5];    // chunks of a tile buffer
  uint64_t kv_empty[2][5];   // value block m's chunk, then the rope chunk (P^T hi)
};
static_assert(sizeof(Bars) <= 272, "barrier block");

// ------------------------------------------------------------------ producers (warps 0-3)
// Warp pw gathers rows 32 pw .. 32 pw + 31 of each tile, chunk by chunk (an instruction moves 4
// rows x 128 bytes, of the rope chunk 8 x 64) in the order in which the values of the tile
// before last release them.  A warp waits for a place and for nothing else: its copies arrive
// on the chunk's barrier when they land, and the score issuer, which waits there, fences them
// for the async proxy.  (With the warps waiting for each tile's copies a tile took two trips
// to L2 in a row.  Prefetching rows to L2 a tile or two ahead costs 8-25% here, and 2% from a warp
// of its own (in bulk; 37% line by line): the copies of two tiles are in flight as it is.  TMA
// tile copies where a warp's rows sit in consecutive slots
// gained 1% there, 2195 to 2173 us, and cost scattered rows 3-9%.)
__device__ void producer(const Problem& p, const CUtensorMap* tm_q, const CUtensorMap* tm_qr,
                         unsigned char* sm, Bars* bars, volatile int* abort, Walk wk) {
  const int lane = threadIdx.x & 31, pw = threadIdx.x >> 5;
  const uint32_t q_base = ptx::smem_addr(sm + kQOff), kv_base = ptx::smem_addr(sm + kKvOff);
  // this lane's place in its warp's rows 4i + lane / 8 (i even, odd) and, of the rope chunk,
  // 8i + lane / 4
  const uint32_t sw_even = pw * (kChunk / 4) + swz(lane >> 3, lane & 7);
  const uint32_t sw_odd = pw * (kChunk / 4) + swz(4 + (lane >> 3), lane & 7);
  const uint32_t sw_rope = pw * (kRopeChunk / 4) + swz64(lane >> 2, lane & 3);
  const unsigned char* kv = (const unsigned char*)p.kv;
  const int64_t q_first = p.qo_indptr[0];
  uint32_t tl = 0, sc = 0;
  bool ok = true;
  Seg s;
  while (ok && next_segment(p, wk, s)) {
    // Slots are read two tiles ahead and scales one, so that neither is waited for: lane holds
    // row 32 pw + lane of the tile in slot / scale, of the next in next / nscale, and the next
    // but one's index, just loaded, in raw (looked at one tile later; a test right after the
    // load cost 1700 clocks a tile).
    int32_t slot, next = -1, raw = -1;
    float scale, nscale = 0.f;
    const int64_t row0 = 32 * pw + lane;
    auto load_raw = [&](int64_t j) {
      const int64_t c = j * kTile + row0;
      if ((j + 1) * kTile <= s.ri.P) raw = p.kv_indices[s.ri.kv_base + c];   // prefix rows only
      else raw = c < s.ri.L ? (int32_t)key_slot(p, s.ri, c) : -1;
    };
    auto take_raw = [&]() {   // -1: no key of the request, or a slot outside the pool
      next = raw >= 0 && raw < p.num_slots ? raw : -1;
      nscale = p.scales[next >= 0 ? next >> p.scale_shift : 0];
    };
    load_raw(s.tile0);
    if (pw == 0) {
      if (sc > 0) {
        int w = lane == 0 ? wait_bar(&bars->q_empty, (sc - 1) & 1, abort, p.wait_ns) : 0;
        ok = __shfl_sync(0xffffffffu, w, 0) != 0;
        if (!ok) break;
      }
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&bars->q_full, kTileBytes);
        const int32_t r0 = (int32_t)((s.r - q_first) * p.heads), r1 = r0 + (int32_t)p.q_rows;
        for (int c = 0; c < 4; ++c) {
          ptx::tma_load_2d(q_base + c * kChunk, tm_q, c * 128, r0, &bars->q_full);
          ptx::tma_load_2d(q_base + c * kChunk + kChunk / 2, tm_q, c * 128, r1, &bars->q_full);
        }
        ptx::tma_load_2d(q_base + 4 * kChunk, tm_qr, 512, r0, &bars->q_full);
        ptx::tma_load_2d(q_base + 4 * kChunk + kRopeChunk / 2, tm_qr, 512, r1, &bars->q_full);
      }
    }
    ++sc;
    take_raw();
    if (s.tile0 + 1 < s.tile1) load_raw(s.tile0 + 1);
    for (int64_t j = s.tile0; j < s.tile1; ++j, ++tl) {
      const uint32_t buf = tl & 1;
      const uint32_t dst = kv_base + buf * kTileBytes;
      slot = next;
      scale = nscale;
      if (j + 1 < s.tile1) {
        take_raw();
        if (j + 2 < s.tile1) load_raw(j + 2);
      }
      auto place = [&](int group) {   // the chunk's place in the buffer is free
        if (tl < 2) return true;
        int w = lane == 0 ? wait_bar(&bars->kv_empty[buf][group], ((tl >> 1) - 1) & 1, abort, p.wait_ns) : 0;
        return __shfl_sync(0xffffffffu, w, 0) != 0;
      };
      // The rows' addresses once for all four chunks; a row that is no key is filled with zeros.
      const unsigned char* mine = kv + (int64_t)max(slot, 0) * q8::kRow;
      const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0);
      const uint32_t live16 = (live >> (lane >> 3)) << 4;     // bit 4 + 4i: row 4i + lane / 8
      const unsigned char* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) src[i] = shfl_ptr(mine, 4 * i + (lane >> 3)) + 16 * (lane & 7);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (ok) ok = place(c);
        if (ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            ptx::cp_async16(dst + c * kChunk + (i >> 1) * 1024 + (i & 1 ? sw_odd : sw_even), src[i] + c * 128,
                            i == 7 ? live >> (28 + (lane >> 3)) << 4 & 16u : (live16 >> (4 * i)) & 16u);
          cp_async_arrive(&bars->kv_full[buf][c]);
        }
      }
      if (ok) ok = place(4);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ptx::cp_async16(dst + 4 * kChunk + i * 512 + sw_rope,
                        shfl_ptr(mine, 8 * i + (lane >> 2)) + 512 + 16 * (lane & 3),
                        ((live >> (8 * i + (lane >> 2))) & 1u) << 4);
      cp_async_arrive(&bars->kv_full[buf][4]);
      // an invalid scale becomes 0: the softmax takes the key as masked
      const bool fine = q8::scale_ok(scale);
      if (slot < 0 && j * kTile + row0 < s.ri.L) raise_error(p, kErrBadSlot);
      if (slot >= 0 && !fine) raise_error(p, kErrBadScale);
      ((float*)(sm + kScaleOff))[buf * 128 + row0] = slot >= 0 && fine ? scale : 0.f;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->sc_full[buf]);
    }
  }
  if (!ok && lane == 0) fail(p, abort);
  ptx::cp_async_commit();
  ptx::cp_async_wait<0>();                // this thread's copies have landed before the CTA exits
  if (pw == 0 && lane == 0 && sc > 0) {   // and q's
    volatile int never = 0;
    ptx::mbar_wait(&bars->q_full, (sc - 1) & 1, &never, 100000000ull);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issuers (warps 12, 13, lane 0)
// Every MMA that this thread issued is done before TMEM is released (bounded wait): also after
// a walk without a timeout, since another role may have had one and not wait for them.
__device__ __forceinline__ void drain_mmas(uint64_t* bar) {
  volatile int never = 0;
  ptx::mma_commit(bar);
  ptx::mbar_wait(bar, 0, &never, 100000000ull);
}

// Scores of each tile, chunk by chunk as its rows land.  Operands are K-major: 32 dims are
// +32 bytes.
__device__ void score_issuer(const Problem& p, unsigned char* sm, Bars* bars, volatile int* abort,
                             uint32_t tmem, Walk wk) {
  const uint32_t q_lo = desc_lo(ptx::smem_addr(sm + kQOff), 16);
  uint32_t tl = 0, sc = 0;
  Seg s;
  while (next_segment(p, wk, s)) {
    if (!spin_bar(&bars->q_full, sc & 1, abort, p.wait_ns)) goto failed;
    for (int64_t j = s.tile0; j < s.tile1; ++j, ++tl) {
      const uint32_t buf = tl & 1, par = (tl >> 1) & 1, d = tmem + kSCol + 128 * buf;
      const uint32_t k_lo = desc_lo(ptx::smem_addr(sm + kKvOff + buf * kTileBytes), 16);
      // the softmax has read the scores of the tile before last
      if (tl >= 2 && !spin_bar(&bars->s_free[buf], par ^ 1, abort, p.wait_ns)) goto failed;
#pragma unroll 1
      for (uint32_t c = 0; c < 5; ++c) {
        if (!spin_bar(&bars->kv_full[buf][c], par, abort, p.wait_ns)) goto failed;
        ptx::fence_proxy_async();   // the copies, for the MMAs of this product and of the values
        ptx::tc_fence_after();
        const uint32_t off = (c * kChunk) >> 4, hi = c < 4 ? kDescSw128 : kDescSw64;
        mma_e4m3(d, k_lo + off, 0, hi, q_lo + off, 0, hi, kIdescQK, c > 0);
        mma_e4m3(d, k_lo + off, 2, hi, q_lo + off, 2, hi, kIdescQK, 1);
        if (c == 4) break;          // 64 rope dims
        mma_e4m3(d, k_lo + off, 4, hi, q_lo + off, 4, hi, kIdescQK, 1);
        mma_e4m3(d, k_lo + off, 6, hi, q_lo + off, 6, hi, kIdescQK, 1);
      }
      ptx::mma_commit(&bars->s_full[buf]);
      if (j + 1 == s.tile1) ptx::mma_commit(&bars->q_empty);
    }
    ++sc;
  }
  drain_mmas(&bars->drain[0]);
  return;
failed:
  fail(p, abort);
  drain_mmas(&bars->drain[0]);
}

// Values of each tile once the softmax has written P^T (and, for a segment's first tile, the
// epilogue before has read O^T); each value block releases its chunk.  Operands are MN-major:
// 32 keys are +4096 (P: 2048) bytes.
__device__ void value_issuer(const Problem& p, unsigned char* sm, Bars* bars, volatile int* abort,
                             uint32_t tmem, Walk wk) {
  const uint32_t lo_lo = desc_lo(ptx::smem_addr(sm + kPLoOff), kRopeChunk);
  uint32_t tl = 0, sc = 0;
  Seg s;
  while (next_segment(p, wk, s)) {
    for (int64_t j = s.tile0; j < s.tile1; ++j, ++tl) {
      if (!spin_bar(&bars->p_full, tl & 1, abort, p.wait_ns)) goto failed;
      const bool first = j == s.tile0;
      if (first && sc > 0 && !spin_bar(&bars->o_free, (sc - 1) & 1, abort, p.wait_ns)) goto failed;
      ptx::tc_fence_after();
      const uint32_t buf = tl & 1, tile = ptx::smem_addr(sm + kKvOff + buf * kTileBytes);
      const uint32_t v_lo = desc_lo(tile, kChunk), hi_lo = desc_lo(tile + 4 * kChunk, kRopeChunk);
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        const uint32_t vm = v_lo + ((m * kChunk) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t voff = (ks * 4096) >> 4, poff = (ks * 2048) >> 4;
          mma_e4m3(tmem + 64 * m, vm, voff, kDescSw128, hi_lo, poff, kDescSw64, kIdescPV4, ks > 0 || !first);
          mma_e4m3(tmem + 64 * m, vm, voff, kDescSw128, lo_lo, poff, kDescSw64, kIdescPV5, 1);
        }
        ptx::mma_commit(&bars->kv_empty[buf][m]);
      }
      ptx::mma_commit(&bars->kv_empty[buf][4]);
      ptx::mma_commit(&bars->pv_done);
      if (j + 1 == s.tile1) ptx::mma_commit(&bars->o_done);
    }
    ++sc;
  }
  drain_mmas(&bars->drain[1]);
  return;
failed:
  fail(p, abort);
  drain_mmas(&bars->drain[1]);
}

// ------------------------------------------------------------------ softmax (warps 4-11)
// NaN codes of 16 bytes become zeros.
__device__ __forceinline__ uint32_t scrub4(uint32_t w) {
  const uint32_t nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  return w & ~nan;
}

// Two weights (P, at most 2^12) as the sums of an e4m3 value (codes in the low 16 bits of hi) and
// an e5m2 value (codes in bytes 1 and 3 of lo: e5m2 is the upper byte of f16).  From 1 up e5m2
// takes the coarse part and e4m3, whose range ends at 448, what is left of it (at most 2^8);
// below, e4m3 takes the coarse part.  What e4m3 leaves is rounded to e5m2 to nearest by adding
// half of its last step, or where P is below 2^-6 by adding the random offset of `dither`.
__device__ __forceinline__ void split_weights(__half2 y, uint32_t dither, uint32_t& hi, uint32_t& lo) {
  const uint32_t coarse = (*(const uint32_t*)&y + 0x00800080u) & 0xff00ff00u & __hge2_mask(y, __float2half2_rn(1.f));
  const __half2 rest = __hsub2(y, *(const __half2*)&coarse);
  hi = q8::pack2(*(const uint32_t*)&rest);
  const uint32_t back = q8::unpack2(hi);
  const __half2 left = __hsub2(y, *(const __half2*)&back);
  const uint32_t small = __hlt2_mask(y, __float2half2_rn(0x1p-6f));
  lo = *(const uint32_t*)&left + ((dither & small) | (0x00800080u & ~small));
}

// ---- merging a column group's partials ----
// out = sum_s w_s o_s, w_s = e^{lse_s - M} / sum, as merge_token() in mtv_common.cuh, but in
// eight slices of eight columns that several CTAs take in turn.  One CTA reads partials at about
// 50 GB/s, and ten of them are 1.3 MB: merged by one CTA they were the last 25-30 us of a batch
// of few long requests.  Who merges:
// - a CTA with more segments to do that finds every other piece done and no one waiting merges
//   straight from its O^T in TMEM, without writing its partial (fast_merge);
// - a CTA without takes its ticket as a helper (kHelper in the group's counter), waits for the
//   other pieces and takes slices until none is left; the CTA of the last piece leaves the merge
//   to helpers where there are any, and takes the slices itself where there are none.
// A helper gives up after p.help_ns (40 us), in one atomic step with looking whether the group is done,
// so that a merge is never left to no one.  (The CTAs of a call need not all be on the GPU at
// once, beside another kernel's; the limit is then what waiting costs.)  A column's bits do not
// depend on who merges it.
constexpr int kHelper = 1 << 16;           // tok_done: finished pieces below, helpers above
// From this many pieces on, CTAs without work help.  A merge of two from TMEM takes 6 us, and a
// helper would have to write its piece first (two: the same times);
// three or four alone took 15-19 us after the last piece (three against five: 64 decoding
// requests 95.3 us a call against 100.7, bs 8, 1k-4k 76.0 against 79.4, bs 32 with 8 heads 86.3
// against 91.5).
constexpr int kHelpPieces = 3;
constexpr int kSlices = 8;
constexpr int kSliceCols = kHeads / kSlices;
static_assert(kSliceCols * 32 == kSoftmaxThreads, "a warp a column for the weights");

// By one warp: the weights of a column into w[s * stride] and its lse to lse_out (or nowhere),
// from the lse of its partials lane and lane + 32 (-inf where there is none).  A NaN partial
// makes them NaN.
__device__ __forceinline__ void column_weights(const float (&l)[2], int nseg, float* w, int stride,
                                               float* lse_out) {
  const int lane = threadIdx.x & 31;
  float e[2];
  float M = fmaxf(l[0], l[1]);
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const float m0 = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int k = 0; k < 2; ++k) e[k] = expf(l[k] - m0);    // 0 for -inf
  float S = e[0] + e[1];
#pragma unroll
  for (int d = 16; d; d >>= 1) S += __shfl_xor_sync(0xffffffffu, S, d);
  const float inv = S == 0.f ? 0.f : 1.f / S;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 32 * k < nseg) w[(lane + 32 * k) * stride] = e[k] * inv;
  if (lane == 0 && lse_out) *lse_out = S == 0.f ? -INFINITY : m0 + logf(S);
}

// The same for all 64 columns of at most kMergeGroup partials, by a thread a column (t < 64), in
// the same order of sums: into w[s][column].
__device__ __forceinline__ void few_weights(const Problem& p, const int32_t* slots, int nseg, int t, float* w,
                                            float* lse_out) {
  float e[kMergeGroup];
#pragma unroll
  for (int k = 0; k < kMergeGroup; ++k)
    e[k] = k < nseg ? __ldcg(p.part_lse + (int64_t)slots[k] * kHeads + t) : -INFINITY;
  float M = e[0];
#pragma unroll
  for (int k = 1; k < kMergeGroup; ++k) M = fmaxf(M, e[k]);
  const float m0 = M == -INFINITY ? 0.f : M;
  float s[kMergeGroup];
#pragma unroll
  for (int k = 0; k < kMergeGroup; ++k) s[k] = e[k] = k < nseg ? expf(e[k] - m0) : 0.f;
#pragma unroll
  for (int d = kMergeGroup / 2; d; d >>= 1)
#pragma unroll
    for (int k = 0; k < d; ++k) s[k] += s[k + d];
  const float inv = s[0] == 0.f ? 0.f : 1.f / s[0];
#pragma unroll
  for (int k = 0; k < kMergeGroup; ++k)
    if (k < nseg) w[k * kHeads + t] = e[k] * inv;
  if (lse_out) *lse_out = s[0] == 0.f ? -INFINITY : m0 + logf(s[0]);
}

// The weights of at most kMergeGroup partials are computed once, of more slice by slice; the
// ticket of the next slice is on its way while a slice's partials are.
__device__ __forceinline__ void merge_slices(const Problem& p, unsigned char* sm, const int32_t* slots, int nseg,
                                             int64_t tok, int64_t lrow0, int ncols, bool alone) {
  const int t = (int)threadIdx.x - kFirstSoftmaxThread, w = t >> 5;
  float* wbuf = (float*)(sm + kWOff);               // [nseg <= 16][64 columns] or [nseg <= 64][8]
  float* lse_s = (float*)(sm + kRedOff);
  volatile int* ticket_s = (volatile int*)(sm + kMiscOff + 16);   // two, in turn
  const bool few = nseg <= kMergeGroup;
  if (few && t < kHeads) few_weights(p, slots, nseg, t, wbuf, lse_s + t);
  if (t == kHeads) ticket_s[0] = alone ? 0 : atomicAdd(p.grp_done + tok * kMergeFan, 1);
  for (int n = 0;; ++n) {
    ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
    const int sl = ticket_s[n & 1];
    if (sl >= kSlices) return;
    int next = 0;
    if (t == kHeads) next = alone ? sl + 1 : atomicAdd(p.grp_done + tok * kMergeFan, 1);
    const int h0 = kSliceCols * sl;
    if (few) {
      if (t < kSliceCols && h0 + t < ncols) p.lse[lrow0 + h0 + t] = lse_s[h0 + t];
    } else {
      const int h = h0 + w, lane = t & 31;
      float l[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        l[k] = lane + 32 * k < nseg ? __ldcg(p.part_lse + (int64_t)slots[lane + 32 * k] * kHeads + h) : -INFINITY;
      column_weights(l, nseg, wbuf + w, kSliceCols, h < ncols ? p.lse + lrow0 + h : nullptr);
      ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
    }
    // float4 4 * 256 sl + 256 e + t of each partial: columns 8 sl + 2 e + t / 128
    float4 acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* at = (const float4*)p.part_o + (4 * sl) * kSoftmaxThreads + t;
    const int stride = few ? kHeads : kSliceCols;
    const float* wt = wbuf + (few ? h0 : 0) + (t >> 7);
#pragma unroll 2
    for (int sg = 0; sg < nseg; sg += 2) {     // pairs, an odd last one with itself, weight 0
      const bool two = sg + 1 < nseg;
      const float4* a0 = at + (int64_t)slots[sg] * (kHeads * kDv / 4);
      const float4* a1 = at + (int64_t)slots[two ? sg + 1 : sg] * (kHeads * kDv / 4);
      float4 v0[4], v1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v0[e] = __ldcg(a0 + e * kSoftmaxThreads);
        if (two) v1[e] = __ldcg(a1 + e * kSoftmaxThreads);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!two) v1[e] = v0[e];
        const float w0 = wt[sg * stride + 2 * e], w1 = two ? wt[(sg + 1) * stride + 2 * e] : 0.f;
        acc[e].x = merge_step(acc[e].x, w0, v0[e].x, w1, v1[e].x);
        acc[e].y = merge_step(acc[e].y, w0, v0[e].y, w1, v1[e].y);
        acc[e].z = merge_step(acc[e].z, w0, v0[e].z, w1, v1[e].z);
        acc[e].w = merge_step(acc[e].w, w0, v0[e].w, w1, v1[e].w);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = (4 * sl + e) * kSoftmaxThreads + t;
      if ((i >> 7) < ncols)
        ((uint2*)(p.out + lrow0 * kDv))[i] =
            make_uint2(ptx::pack_bf16x2(acc[e].x, acc[e].y), ptx::pack_bf16x2(acc[e].z, acc[e].w));
    }
    if (t == kHeads) ticket_s[(n + 1) & 1] = next;
  }
}

// One thread of a helper: whether it is to merge.
__device__ __forceinline__ bool help_merge(const Problem& p, int* counter, int nseg, volatile int* abort) {
  const uint64_t t0 = ptx::globaltimer();
  while ((ptx::ld_acquire_gpu(counter) & (kHelper - 1)) < nseg) {
    if (*abort || ptx::globaltimer() - t0 >= p.help_ns) {
      atomicAdd(&p.hdr->helps_left, 1u);
      return (atomicSub(counter, kHelper) & (kHelper - 1)) == nseg;
    }
    __nanosleep(100);
  }
  atomicAdd(&p.hdr->helps, 1u);
  return true;
}

// kGT: draft tokens per group of 64 columns (1 for 64 heads per token, 8 for 8 heads).
//
// A wait that gives up marks the thread (dead) and the CTA (abort) and the thread goes on
// without waiting, to the end of its walk, so that every thread still meets the named
// barriers; the outputs of such a call are not valid (MLA_TV_DEV_TIMEOUT).
template <int kGT>
__device__ void softmax_role(const Problem& p, unsigned char* sm, Bars* bars, volatile int* abort,
                             uint32_t tmem, Walk wk) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t quarter = warp & 3;               // TMEM lanes 32*quarter .. +31
  const uint32_t half = (warp - kProducerWarps) >> 2;   // columns [32*half, 32*half + 32)
  const uint32_t hb = 32 * half;
  const uint32_t row = 32 * quarter + lane;        // key row of the tile / value dim in a block
  const uint32_t tl_lane = (32u * quarter) << 16;
  float* red = (float*)(sm + kRedOff);             // [4 quarters][64 columns]; at the end [64][4]
  float* nref_s = (float*)(sm + kRefOff);
  float* factor_s = (float*)(sm + kFactorOff);
  float* inv_l = (float*)(sm + kInvLOff);
  volatile int* ticket_s = (volatile int*)(sm + kMiscOff + 16);
  int32_t* slots_s = (int32_t*)(sm + kSlotOff);
  SegInfo* si = (SegInfo*)(sm + kSegOff);
  const int64_t q_first = p.qo_indptr[0];
  uint32_t tl = 0, sc = 0;
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !wait_bar(bar, parity, abort, p.wait_ns)) {
      dead = true;
      fail(p, abort);
    }
  };
  Seg s;
  while (next_segment(p, wk, s)) {
    if (threadIdx.x == kFirstSoftmaxThread) {   // read back in the epilogue, after barriers
      si->map = s.map;
      si->nseg = s.nseg;
      si->piece = s.piece;
      si->seg = s.seg;
    }
    float lp[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) lp[i] = 0.f;
    float m_ref = kNoKey;     // quarter 0: column hb + lane's reference
    if (quarter == 0) {
      const int col = (int)hb + lane;
      factor_s[col] = col < s.ncols ? p.q_factor[(s.r - q_first) * p.heads + col] : 0.f;
      nref_s[col] = -kNoKey;
    }
    // Also: the epilogue before has read its scratch, P^T lo may be written again.
    ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
    for (int64_t j = s.tile0; j < s.tile1; ++j, ++tl) {
      const uint32_t buf = tl & 1, par = (tl >> 1) & 1;
      unsigned char* tile = sm + kKvOff + buf * kTileBytes;
      const int64_t c = j * kTile + row;
      // Which of this thread's columns see key c, by the mask alone: one token for 64 heads
      // per token; with 8 heads, bit q of vq for the token of columns hb + 8q .. hb + 8q + 7.
      uint32_t vq = 0u;
      if constexpr (kGT == 1) {
        vq = c < s.ri.L && key_visible(p, s.ri, s.t, c) ? 15u : 0u;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int32_t col = (int32_t)hb + 8 * q;
          if (c < s.ri.L && col < s.ncols && key_visible(p, s.ri, kGT * s.t + (col >> 3), c)) vq |= 1u << q;
        }
      }
      wait(&bars->sc_full[buf], par);
      const float g = ((const float*)(sm + kScaleOff))[buf * 128 + row];   // 0: no valid key
      if (!(g > 0.f)) vq = 0u;
      float lg = g > 0.f ? __log2f(g) : 0.f, inv_g = g > 0.f ? __frcp_rn(g) : 0.f;
      // y less the reference is (hi + lo) u + v; u and v while the scores are not there yet
      uint64_t u2[16], v2[16];
      {
        const uint64_t g2 = ptx::pack_f32x2(g, g), lg2 = ptx::pack_f32x2(lg, lg);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ulonglong2 f = *(const ulonglong2*)(factor_s + hb + 4 * i);
          const ulonglong2 n = *(const ulonglong2*)(nref_s + hb + 4 * i);
          u2[2 * i] = ptx::mul_f32x2(f.x, g2);
          u2[2 * i + 1] = ptx::mul_f32x2(f.y, g2);
          v2[2 * i] = ptx::add_f32x2(n.x, lg2);
          v2[2 * i + 1] = ptx::add_f32x2(n.y, lg2);
        }
      }
      // random bits of the key column, for the rounding of small weights (split_weights)
      uint32_t dither = (uint32_t)c * 0x9e3779b1u;
      dither = (dither ^ (dither >> 16)) * 0x9e3779b1u;
      dither = (dither >> 24) | (dither & 0x00ff0000u);
      wait(&bars->s_full[buf], par);
      __syncwarp();
      ptx::tc_fence_after();
      float x[32];     // P's exponents
      const uint32_t ts = tmem + tl_lane + kSCol + 128 * buf + hb;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi[16], lo[16];
        ptx::tmem_ld16(ts + 16 * h, hi);
        ptx::tmem_ld16(ts + 64 + 16 * h, lo);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t t = ptx::add_f32x2(ptx::pack_u32x2(hi[2 * i], hi[2 * i + 1]),
                                            ptx::pack_u32x2(lo[2 * i], lo[2 * i + 1]));
          ptx::unpack_f32x2(ptx::fma_f32x2(t, u2[8 * h + i], v2[8 * h + i]), x[16 * h + 2 * i], x[16 * h + 2 * i + 1]);
        }
      }
      if (__builtin_expect(__any_sync(0xffffffffu, vq != 15u), 0)) {
        // A NaN code in a row that some column must not see would reach it through 0 x NaN in
        // the value product: such a row's scores are NaN, and its NaN codes are zeroed here
        // (columns that see the row carry NaN weights).  The other half's threads may see no
        // reason to, so all 512 dims are looked at; who does it twice writes the same.
        if (vq != 15u) {
          bool nan = false;
#pragma unroll
          for (int i = 0; i < 32; ++i) nan |= x[i] != x[i];
          if (nan) {
#pragma unroll 1
            for (int gq = 0; gq < 32; ++gq) {
              uint4* at = (uint4*)(tile + (gq >> 3) * kChunk + swz(row, gq & 7));
              uint4 w = *at;
              *at = make_uint4(scrub4(w.x), scrub4(w.y), scrub4(w.z), scrub4(w.w));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!((vq >> (i >> 3)) & 1u)) x[i] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, x[i]);
      // The four warps that share these 32 columns agree on whether a score rose too far
      // above its column's reference (a segment's first keys always do).
      if (__builtin_expect(ptx::bar_any(kHalfBar + half, 128, top > kPBits + kLag), 0)) {
        // A row without values gets the scale 2^-60 in place of its own.
        uint32_t any = vq == 0u;
#pragma unroll 1
        for (int gq = 0; gq < 32 && any == 0u; ++gq) {
          const uint4 w = *(const uint4*)(tile + (gq >> 3) * kChunk + swz(row, gq & 7));
          any = (w.x | w.y | w.z | w.w) & 0x7f7f7f7fu;
        }
        if (any == 0u) {
          lg = -kEmptyBits;
          inv_g = kEmptyInv;
        }
        // New references: each column's exact maximum so far.  Each warp reduces its 32 rows;
        // lane i of the half's quarter-0 warp folds the quarters into column hb + i.
        // y itself: nothing of it is left beside the reference of a column without keys
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi[16], lo[16];
          ptx::tmem_ld16(ts + 16 * h, hi);
          ptx::tmem_ld16(ts + 64 + 16 * h, lo);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const float4 f = *(const float4*)(factor_s + hb + 16 * h + 4 * i4);
            const float fa[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 4 * i4 + i;
              const float t = __uint_as_float(hi[k]) + __uint_as_float(lo[k]);
              x[16 * h + k] = (vq >> ((16 * h + k) >> 3)) & 1u ? fmaf(t, fa[i] * g, lg) : -INFINITY;
            }
          }
        }
        float mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float r = ptx::warp_max(x[i]);
          mine = lane == i ? r : mine;
        }
        red[64 * quarter + hb + lane] = mine;
        ptx::bar_sync(kHalfBar + half, 128);
        if (quarter == 0) {
          const float* at = red + hb + lane;
          const float ref = fmaxf(fmaxf(at[0], at[64]), fmaxf(at[128], at[192])) - kPBits;
          float alpha = 1.f;
          if (ref > m_ref) {
            alpha = m_ref == kNoKey ? 0.f : ptx::ex2(m_ref - ref);
            m_ref = ref;
            nref_s[hb + lane] = -ref;
          }
          red[hb + lane] = alpha;    // over the quarter's own maxima, which no one else reads
        }
        ptx::bar_sync(kHalfBar + half, 128);
#pragma unroll
        for (int i4 = 0; i4 < 8; ++i4) {
          const float4 n = *(const float4*)(nref_s + hb + 4 * i4);
          x[4 * i4] += n.x;
          x[4 * i4 + 1] += n.y;
          x[4 * i4 + 2] += n.z;
          x[4 * i4 + 3] += n.w;
        }
        // l, and once the values of the tile before are done O^T, follow the references, 16
        // columns at a time (warp-uniform: every lane reads the same factors)
        if (j != s.tile0) {
          wait(&bars->pv_done, (tl - 1) & 1);
          __syncwarp();
          ptx::tc_fence_after();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float al[16];
            bool rescale = false;
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              const float4 a4 = *(const float4*)(red + hb + 16 * q + 4 * i4);
              al[4 * i4] = a4.x;
              al[4 * i4 + 1] = a4.y;
              al[4 * i4 + 2] = a4.z;
              al[4 * i4 + 3] = a4.w;
              rescale |= (a4.x != 1.f) | (a4.y != 1.f) | (a4.z != 1.f) | (a4.w != 1.f);
            }
            if (!rescale) continue;
#pragma unroll
            for (int i = 0; i < 16; ++i) lp[16 * q + i] *= al[i];
#pragma unroll 1
            for (int mb = 0; mb < 4; ++mb) {
              uint32_t o[16];
              const uint32_t ta = tmem + tl_lane + hb + 16 * q + 64 * mb;
              ptx::tmem_ld16(ta, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al[i]);
              ptx::tmem_st16(ta, o);
            }
          }
          ptx::tmem_wait_st();
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->s_free[buf]);
      uint32_t phi[8], plo[8];            // P^T of this row, 32 columns
#pragma unroll
      for (int i4 = 0; i4 < 8; ++i4) {
        const float e0 = ptx::ex2(x[4 * i4]), e1 = ptx::ex2(x[4 * i4 + 1]);
        const float e2 = ptx::ex2(x[4 * i4 + 2]), e3 = ptx::ex2(x[4 * i4 + 3]);
        lp[4 * i4] = fmaf(e0, inv_g, lp[4 * i4]);
        lp[4 * i4 + 1] = fmaf(e1, inv_g, lp[4 * i4 + 1]);
        lp[4 * i4 + 2] = fmaf(e2, inv_g, lp[4 * i4 + 2]);
        lp[4 * i4 + 3] = fmaf(e3, inv_g, lp[4 * i4 + 3]);
        uint32_t w[2], v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) split_weights(__floats2half2_rn(k ? e2 : e0, k ? e3 : e1), dither, w[k], v[k]);
        phi[i4] = w[0] | (w[1] << 16);
        plo[i4] = __byte_perm(v[0], v[1], 0x7531);
      }
      unsigned char* hi_dst = tile + 4 * kChunk;
      unsigned char* lo_dst = sm + kPLoOff;
      *(uint4*)(hi_dst + swz64(row, 2 * half)) = make_uint4(phi[0], phi[1], phi[2], phi[3]);
      *(uint4*)(hi_dst + swz64(row, 2 * half + 1)) = make_uint4(phi[4], phi[5], phi[6], phi[7]);
      // P^T lo is free once the values of the tile before are done.
      if (tl > 0) wait(&bars->pv_done, (tl - 1) & 1);
      *(uint4*)(lo_dst + swz64(row, 2 * half)) = make_uint4(plo[0], plo[1], plo[2], plo[3]);
      *(uint4*)(lo_dst + swz64(row, 2 * half + 1)) = make_uint4(plo[4], plo[5], plo[6], plo[7]);
      ptx::fence_proxy_async();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->p_full);
    }
    // epilogue: l across the 128 rows, normalised O^T, lse
    const float l_col = warp_transpose_reduce<false>(lp);
    wait(&bars->o_done, sc & 1);   // every warp is through its last tile, P^T lo is free
    __syncwarp();
    ptx::tc_fence_after();
    red[(hb + lane) * 4 + quarter] = l_col;
    ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
    const int64_t nseg = si->nseg;
    const int32_t seg = si->seg, piece = si->piece;
    {   // the column group's partial slots, read by the merge paths after later barriers
      const int t = (int)threadIdx.x - kFirstSoftmaxThread;
      if (t < nseg) slots_s[t] = (int32_t)si->map.slot(t);
    }
    if (quarter == 0) {  // lane i of the quarter-0 warp of each half finalises column hb + i
      const float4 t4 = *(const float4*)(red + (hb + lane) * 4);
      const float l = (t4.x + t4.y) + (t4.z + t4.w);      // NaN stays NaN
      inv_l[hb + lane] = l == 0.f ? 0.f : 1.f / l;
      const float lse = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
      if (nseg == 1) {
        if ((int32_t)(hb + lane) < s.ncols) p.lse[s.r * p.heads + hb + lane] = lse;
      } else {
        p.part_lse[(int64_t)seg * kHeads + hb + lane] = lse;
      }
    }
    const int64_t tok = s.r - q_first;
    // no helper: more segments to do
    const bool busy = wk.u < wk.u_end || nseg < kHelpPieces || p.merge_mode == 2;
    if (threadIdx.x == kFirstSoftmaxThread)
      *ticket_s = nseg > 1 && nseg <= kMergeGroup && p.merge_mode == 0 &&
                  ptx::ld_acquire_gpu(p.tok_done + tok) == nseg - 1;
    ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
    if (*ticket_s) {   // every other piece is done, none of them by a helper
      float* wb = (float*)(sm + kWOff);
      const int t = (int)threadIdx.x - kFirstSoftmaxThread;
      if (t < kHeads) few_weights(p, slots_s, (int)nseg, t, wb, t < s.ncols ? p.lse + s.r * p.heads + t : nullptr);
      if (t == 0) atomicAdd(&p.hdr->merges_tmem, 1u);
      ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
      fast_merge<1, (kGT > 1)>(p, tmem + tl_lane + hb, s.r * p.heads, s.ncols, slots_s, nseg,
                               (int64_t)piece, hb, row, inv_l, wb);
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bars->o_free);
      ++sc;
      continue;
    }
    const bool whole = nseg == 1;   // its normalised output is final (bf16, RNE)
    uint16_t* dst = p.out + (s.r * p.heads + hb) * kDv + (row & ~3u);
    float* part = p.part_o + ((int64_t)seg * kHeads + hb) * kDv + row;
    const int32_t nvalid = s.ncols - (int32_t)hb;   // of this thread's 32 columns
#pragma unroll 1
    for (int mb = 0; mb < 4; ++mb) {
      uint32_t r16[2][16];
      ptx::tmem_ld16(tmem + tl_lane + 64 * mb + hb, r16[0]);
      ptx::tmem_ld16(tmem + tl_lane + 64 * mb + hb + 16, r16[1]);
      ptx::tmem_wait_ld();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(__uint_as_float(r16[i >> 4][i & 15]), inv_l[hb + i]);
      if (whole) store_heads_bf16<(kGT > 1)>(dst + 128 * mb, v, nvalid);
      else {
#pragma unroll
        for (int i = 0; i < 32; ++i) __stcg(part + i * kDv + 128 * mb, v[i]);
      }
    }
    ptx::tc_fence_before();
    ptx::mbar_arrive(&bars->o_free);
    if (!whole) {
      // Ticket: with the column group's last piece its partials are merged.
      __threadfence();
      ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
      if (threadIdx.x == kFirstSoftmaxThread) {
        int* counter = p.tok_done + tok;
        const int old = atomicAdd(counter, busy ? 1 : kHelper + 1);
        const bool last = (old & (kHelper - 1)) == nseg - 1;
        if (last) atomicAdd(&p.hdr->merges_ws, 1u);
        *ticket_s = busy ? last && old < kHelper : last || help_merge(p, counter, (int)nseg, abort);
      }
      ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
      const bool merge = *ticket_s;
      if (merge) {
        __threadfence();
        ptx::bar_sync(kSoftmaxBar, kSoftmaxThreads);
        merge_slices(p, sm, slots_s, (int)nseg, tok, s.r * p.heads, s.ncols, busy);
      }
    }
    ++sc;
  }
}

template <int kGT>
__global__ void __launch_bounds__(kThreads, 1)
    split_q8_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_qr, const Problem p) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Bars* bars = (Bars*)(sm + kBarOff);
  uint32_t* tmem_slot = (uint32_t*)(sm + kMiscOff);
  volatile int* abort = (volatile int*)(sm + kMiscOff + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars->q_full, 1);
    ptx::mbar_init(&bars->q_empty, 1);
    ptx::mbar_init(&bars->p_full, kSoftmaxWarps);
    ptx::mbar_init(&bars->pv_done, 1);
    ptx::mbar_init(&bars->o_done, 1);
    ptx::mbar_init(&bars->o_free, kSoftmaxThreads);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&bars->drain[b], 1);
      ptx::mbar_init(&bars->s_free[b], kSoftmaxWarps);
      ptx::mbar_init(&bars->sc_full[b], kProducerWarps);
      ptx::mbar_init(&bars->s_full[b], 1);
      for (int g = 0; g < 5; ++g) {
        ptx::mbar_init(&bars->kv_empty[b][g], 1);
        ptx::mbar_init(&bars->kv_full[b][g], 32 * kProducerWarps);
      }
    }
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kValueWarp) ptx::tmem_alloc(tmem_slot, kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The prologue above overlaps the planner; its results are read only after it is done.
  // Meanwhile the first MiB of indices goes to L2, a share a CTA: the first tiles' index loads
  // wait for the plan and are waited for (bs 8, 1k-4k 80.6 -> 78.7 us; 64 decoding requests 100.0
  // -> 97.0; the rows of the first 256 or 1024 indices a CTA as well: no gain to 30% more).
  if (warp == 0) {
    const int64_t i0 = max(p.kv_indptr[0], 0), i1 = min((int64_t)p.kv_indptr[p.bs], p.num_kv_indices);
    const int64_t lines = min((i1 - i0 + 31) >> 5, (int64_t)8192);
    for (int64_t l = (int64_t)blockIdx.x * 32 + lane; l < lines; l += (int64_t)gridDim.x * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.kv_indices + i0 + 32 * l));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Walk wk;
  wk.W = p.lanes;
  wk.g = (int32_t)blockIdx.x / wk.W;
  wk.lane = (int32_t)blockIdx.x - wk.g * wk.W;
  const int64_t C = p.hdr->capacity;
  wk.u = (int64_t)wk.g * C;
  wk.u_end = min(p.hdr->total_units, wk.u + C);
  wk.J = wk.g < p.hdr->groups ? p.grp_job[wk.g] : 0;

  if (wk.g >= p.hdr->groups || wk.u >= wk.u_end) {
    // no work for this CTA
  } else if (ptx::smem_addr(sm) & 1023u) {
    // the swizzles need a 1024-byte aligned base, which dynamic shared memory has
    if (threadIdx.x == 0) raise_error(p, kErrTimeout);
  } else if (warp < kProducerWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    producer(p, &tm_q, &tm_qr, sm, bars, abort, wk);
  } else if (warp >= kScoreWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kScoreWarp && lane == 0) score_issuer(p, sm, bars, abort, tmem, wk);
    if (warp == kValueWarp && lane == 0) value_issuer(p, sm, bars, abort, tmem, wk);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<kGT>(p, sm, bars, abort, tmem, wk);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kValueWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// The split queries as [2 q_rows][576] bytes, box [64 rows][inner bytes].
bool encode_split_q(CUtensorMap* map, const Problem& p, uint32_t inner) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)q8::kRow, (cuuint64_t)(2 * p.q_rows)};
  cuuint64_t strides[1] = {(cuuint64_t)q8::kRow};
  cuuint32_t box[2] = {inner, 64};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.q_split, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tq

cudaError_t split_q8_prepare() {
  cudaError_t e = cudaFuncSetAttribute(tq::split_q8_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)tq::kSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(tq::split_q8_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)tq::kSmemBytes);
}

int launch_split_q8(const Problem& p, int grid, cudaStream_t stream) {
  if (p.total_q <= 0) return 0;
  CUtensorMap tm_q, tm_qr;
  if (!tq::encode_split_q(&tm_q, p, 128) || !tq::encode_split_q(&tm_qr, p, 64)) return -1;
  // Programmatic dependent launch: the kernel's prologue may overlap the planner.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(tq::kThreads);
  cfg.dynamicSmemBytes = tq::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = p.group_tokens == 1
                            ? cudaLaunchKernelEx(&cfg, tq::split_q8_kernel<1>, tm_q, tm_qr, p)
                            : cudaLaunchKernelEx(&cfg, tq::split_q8_kernel<8>, tm_q, tm_qr, p);
  return e == cudaSuccess ? 0 : -1;
}

}  // namespace mtv
