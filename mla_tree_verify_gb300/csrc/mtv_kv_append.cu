// Appending latent-cache rows with the position rotation, and rotating the queries' rope part.
//
// Per token: row = [latent, rot(k_pe)]; written as bf16, or as e4m3 codes of row / scale.
// rot turns pair k = (a, b) by the angle whose (cos, sin) the table holds for the token's
// position: (a c - b s, b c + a s), in fp32; one rounding follows, to the type that is kept.
//
// Layout on the GPU.  The work is bound by HBM bytes (decoding steps of a few tokens by
// latency): a row reads 1152 B and writes 576 or 1152, each query head reads and writes 128.
// One warp does one item, with no shared memory and the item's data loaded before its slot and
// position are looked at (one trip to memory less; a skipped token's data is read for nothing).
// With more than eight query heads, a token's items are its row (lane l holds dims 8l..8l+7 and
// 256+8l..256+8l+7, two 16-byte loads, and rope pair l) and its heads in sixteens.  With fewer,
// such items would hold too few bytes to keep the memory busy: the heads of as many tokens as
// make sixteen are one item, their rows go two to an item.  A token's items are neighbours, so its
// table row is read from DRAM once.  16385 tokens, 64 heads, e4m3: 52.4 us; 32768 tokens, 8
// heads, bf16: 30.9 us (an item a token 36.9, rows alone 34.9, four rows an item 32.6).
#include "mtv_kv_append.cuh"

#include "mtv_common.cuh"
#include "mtv_q8.cuh"

namespace mtv {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kHeadsPerItem = 16;
constexpr int kRowsPerItem = 2;   // with few heads
constexpr int kRopeHalf = 32;
constexpr uint32_t kBadSlot = 1u, kBadPos = 2u, kBadValue = 4u, kBadScale = 8u;

// Not .nc: queries may be rotated in place.
__device__ __forceinline__ uint4 ld16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The slot and position of token i; false (flagged by its row's item): nothing is to be written.
__device__ __forceinline__ bool token(const AppendArgs& a, int64_t i, bool flag, int64_t& slot, int64_t& pos) {
  slot = a.slots[i];
  pos = a.positions[i];
  if (slot == -1) return false;
  const uint32_t bad = (slot < 0 || slot >= a.num_slots ? kBadSlot : 0u) |
                       (pos < 0 || pos >= a.max_pos ? kBadPos : 0u);
  if (bad && flag && (threadIdx.x & 31) == 0) atomicOr(a.status, bad);
  return bad == 0u;
}

// What a row needs from memory but its table entries.
struct RowIn {
  uint4 w0, w1;
  uint16_t ka, kb;
};

template <bool kInter>
__device__ __forceinline__ RowIn load_row(const AppendArgs& a, int64_t i) {
  const int lane = threadIdx.x & 31;
  const uint16_t* src = a.latent + i * a.latent_stride + 8 * lane;
  const uint16_t* kp = a.k_pe + i * a.k_pe_stride;
  RowIn r;
  r.w0 = ld16(src);
  r.w1 = ld16(src + 256);
  r.ka = kp[kInter ? 2 * lane : lane];
  r.kb = kp[kInter ? 2 * lane + 1 : lane + kRopeHalf];
  return r;
}

// kType: MLA_KV_TYPE_*; kGiven: scales are read, not computed; (c, s): lane's pair of the table.
template <int kType, bool kGiven, bool kInter>
__device__ __forceinline__ void append_row(const AppendArgs& a, const RowIn& in, int64_t slot, float c, float s) {
  const int lane = threadIdx.x & 31;
  const uint4 w0 = in.w0, w1 = in.w1;
  const float ra = bf16_to_f32(in.ka), rb = bf16_to_f32(in.kb);
  float x[16];
  widen8(w0, *(float(*)[8])x);
  widen8(w1, *(float(*)[8])(x + 8));
  float ya = ra * c - rb * s, yb = rb * c + ra * s;
  if constexpr (kType == 0) {
    uint16_t* dst = (uint16_t*)a.kv + slot * kDqk;
    *(uint4*)(dst + 8 * lane) = w0;
    *(uint4*)(dst + 256 + 8 * lane) = w1;
    const uint32_t y = bf16x2(ya, yb);
    // an exponent of ones (NaN, infinity) carries into the sign's place
    auto ones = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
    const uint32_t bad = ones(w0.x) | ones(w0.y) | ones(w0.z) | ones(w0.w) | ones(w1.x) | ones(w1.y) |
                         ones(w1.z) | ones(w1.w) | ones(y);
    if (bad & 0x80008000u) atomicOr(a.status, kBadValue);
    if constexpr (kInter) {
      *(uint32_t*)(dst + kDv + 2 * lane) = y;
    } else {
      dst[kDv + lane] = (uint16_t)y;
      dst[kDv + lane + kRopeHalf] = (uint16_t)(y >> 16);
    }
  } else {
    // NaN and infinities: |x| as an integer is at least that of infinity (max keeps it)
    uint32_t top = max(__float_as_uint(ya) & 0x7fffffffu, __float_as_uint(yb) & 0x7fffffffu);
#pragma unroll
    for (int k = 0; k < 16; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    const float amax = __uint_as_float(top);     // NaN if any value is
    float scale;
    bool poison = false;
    if constexpr (kGiven) {
      scale = a.scales[slot >> a.scale_shift];
      if (!q8::scale_ok(scale)) {
        if (lane == 0) atomicOr(a.status, kBadScale);
        return;
      }
      if (top >= 0x7f800000u) {   // infinities become NaN: saturated, they would look like values
        if (lane == 0) atomicOr(a.status, kBadValue);
        auto drop = [](float v) { return v - v == 0.f ? v : __uint_as_float(0x7fffffffu); };
        ya = drop(ya);
        yb = drop(yb);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = drop(x[k]);
      }
    } else {
      scale = amax > 0.f ? fmaxf(amax * (1.f / q8::kMax), q8::kScaleMin) : 1.f;
      poison = !(amax <= q8::kMax * q8::kScaleMax);
      if (poison) scale = 1.f;
      if (lane == 0) {
        if (poison) atomicOr(a.status, kBadValue);
        a.scales[slot] = scale;
      }
    }
    const float inv = __frcp_rn(scale);
    uint32_t z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      z[k] = poison ? q8::kNanCode4
                    : q8::pack4(x[4 * k] * inv, x[4 * k + 1] * inv, x[4 * k + 2] * inv,
                                x[4 * k + 3] * inv);
    uint8_t* dst = (uint8_t*)a.kv + slot * q8::kRow;
    *(uint2*)(dst + 8 * lane) = make_uint2(z[0], z[1]);
    *(uint2*)(dst + 256 + 8 * lane) = make_uint2(z[2], z[3]);
    const uint32_t y = poison ? q8::kNanCode4 : q8::pack2(ya * inv, yb * inv);
    if constexpr (kInter) {
      *(uint16_t*)(dst + kDv + 2 * lane) = (uint16_t)y;
    } else {
      dst[kDv + lane] = (uint8_t)y;
      dst[kDv + lane + kRopeHalf] = (uint8_t)(y >> 8);
    }
  }
}

// Rows [i, min(i + kRows, end)).
template <int kType, bool kGiven, bool kInter, int kRows>
__device__ __forceinline__ void append_rows(const AppendArgs& a, int64_t i, int64_t end) {
  const int lane = threadIdx.x & 31;
  RowIn in[kRows];
  bool live[kRows];
  int64_t slot[kRows], pos[kRows];
  float c[kRows], s[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (i + k < end) in[k] = load_row<kInter>(a, i + k);
#pragma unroll
  for (int k = 0; k < kRows; ++k) live[k] = i + k < end && token(a, i + k, true, slot[k], pos[k]);
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (live[k]) {
      c[k] = a.cos_sin[pos[k] * 64 + lane];
      s[k] = a.cos_sin[pos[k] * 64 + kRopeHalf + lane];
    }
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (live[k]) append_row<kType, kGiven, kInter>(a, in[k], slot[k], c[k], s[k]);
}

// Sixteen heads' queries, so that no value crosses lanes.  Interleaved: eight lanes a head, 16
// bytes each (with 32 bytes of four lanes instead, 16385 tokens of 64 heads took 60 us against
// 53); halves: four lanes a head, 16 bytes of each half (with a shuffle between eight lanes,
// 32768 tokens of 8 heads took 32 us against 29).  Slot j of the sixteen is head h0 + j of token
// i, or with kMany (heads <= 8) head j % heads of token i + j / heads.
template <bool kGiven, bool kInter, bool kMany>
__device__ __forceinline__ void rotate_heads(const AppendArgs& a, int64_t i, int h0) {
  constexpr int kLanes = kInter ? 8 : 4, kParts = kInter ? 1 : 2;   // lanes a head, loads a lane
  constexpr int kHeads = 32 / kLanes, kRounds = kHeadsPerItem / kHeads, kPairs = 4 * kParts;
  constexpr int kTables = kMany ? kRounds : 1;                      // tokens a lane meets
  const int lane = threadIdx.x & 31, g = lane & (kLanes - 1), sub = lane / kLanes;
  uint4 w[kRounds][kParts];
  int64_t tok[kRounds];
  int head[kRounds];
  bool on[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int j = kHeads * k + sub;
    const int up = kMany ? j / a.heads : 0;
    tok[k] = i + up;
    head[k] = kMany ? j - up * a.heads : h0 + j;
    on[k] = kMany ? up < (int)a.bundle && tok[k] < a.n : head[k] < a.heads;
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      if (on[k]) w[k][q] = ld16(a.q_pe + tok[k] * a.q_ts + head[k] * a.q_hs + 8 * g + kRopeHalf * q);
  }
  float c[kTables][kPairs], s[kTables][kPairs];
  bool live[kTables];
  int64_t slot[kTables], pos[kTables];
#pragma unroll
  for (int k = 0; k < kTables; ++k)
    live[k] = (!kMany || on[k]) && token(a, tok[k], false, slot[k], pos[k]) &&
              (!kGiven || q8::scale_ok(a.scales[slot[k] >> a.scale_shift]));
#pragma unroll
  for (int k = 0; k < kTables; ++k) {
    if (!live[k]) continue;
    const float* cs = a.cos_sin + pos[k] * 64 + kPairs * g;
#pragma unroll
    for (int q = 0; q < kPairs; q += 4) {
      *(float4*)(c[k] + q) = *(const float4*)(cs + q);
      *(float4*)(s[k] + q) = *(const float4*)(cs + kRopeHalf + q);
    }
  }
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    constexpr int kOne = kMany ? 1 : 0;
    const int t = k * kOne;
    if (!on[k] || !live[t]) continue;
    float x[8 * kParts], y[8 * kParts];
#pragma unroll
    for (int q = 0; q < kParts; ++q) widen8(w[k][q], *(float(*)[8])(x + 8 * q));
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const int ia = kInter ? 2 * q : q, ib = kInter ? 2 * q + 1 : q + 8;
      y[ia] = x[ia] * c[t][q] - x[ib] * s[t][q];
      y[ib] = x[ib] * c[t][q] + x[ia] * s[t][q];
    }
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      *(uint4*)(a.q_out + tok[k] * a.o_ts + head[k] * a.o_hs + 8 * g + kRopeHalf * q) =
          make_uint4(bf16x2(y[8 * q], y[8 * q + 1]), bf16x2(y[8 * q + 2], y[8 * q + 3]),
                     bf16x2(y[8 * q + 4], y[8 * q + 5]), bf16x2(y[8 * q + 6], y[8 * q + 7]));
  }
}

template <int kType, bool kGiven, bool kInter, bool kMany>
__global__ void __launch_bounds__(kAppendThreads, kMany ? 4 : kInter ? 6 : 5)
    kv_append_kernel(const AppendArgs a) {
  const uint32_t item = blockIdx.x * (uint32_t)(kAppendThreads / 32) + (threadIdx.x >> 5);
  if (item >= a.items) return;
  const uint32_t group = item / a.parts, part = item - group * a.parts;
  const int64_t i = (int64_t)group * a.bundle;
  constexpr int kRows = kMany ? kRowsPerItem : 1;
  const uint32_t row_items = (a.bundle + kRows - 1) / kRows;
  if (part < row_items) {
    append_rows<kType, kGiven, kInter, kRows>(a, i + part * kRows, min((int64_t)a.n, i + a.bundle));
  } else {
    rotate_heads<kGiven, kInter, kMany>(a, i, (part - row_items) * kHeadsPerItem);
  }
}

template <int kType, bool kGiven>
void launch_inter(const AppendArgs& a, bool inter, unsigned grid, cudaStream_t st) {
  if (a.bundle > 1) {
    if (inter) kv_append_kernel<kType, kGiven, true, true><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<kType, kGiven, false, true><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    if (inter) kv_append_kernel<kType, kGiven, true, false><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<kType, kGiven, false, false><<<grid, kAppendThreads, 0, st>>>(a);
  }
}

}  // namespace

AppendShape kv_append_shape(int64_t n, int32_t heads) {
  AppendShape s;
  if (heads > kHeadsPerItem / 2) {
    s.bundle = 1;
    s.parts = 1 + (heads + kHeadsPerItem - 1) / kHeadsPerItem;
  } else {
    s.bundle = heads ? kHeadsPerItem / heads : kRowsPerItem;
    s.parts = (s.bundle + kRowsPerItem - 1) / kRowsPerItem + (heads ? 1 : 0);
  }
  s.items = (n + s.bundle - 1) / s.bundle * s.parts;
  return s;
}

int launch_kv_append(const AppendArgs& a, int type, bool given, bool inter, cudaStream_t stream) {
  const int64_t warps = kAppendThreads / 32;
  const unsigned grid = (unsigned)((a.items + warps - 1) / warps);
  if (type == 0) launch_inter<0, false>(a, inter, grid, stream);
  else if (given) launch_inter<1, true>(a, inter, grid, stream);
  else launch_inter<1, false>(a, inter, grid, stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mtv
