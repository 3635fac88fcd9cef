// attention.hip -- attention of new tokens over the paged cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp2(c q . k_j - m),   c = scale * log2(e)
//
// in one pass over the keys: a running maximum m and sum of each row, and the
// rows of the output rescaled when m has grown by more than 2^kSlack.  Weights
// that are rounded to fp16, whose steps end at 2^-24, are kept 2^kLift larger (m
// lies that far below the maximum): at most 2^15, so none overflows, and the
// fixed steps begin at 2^-21 of the largest weight and are 2^-31 of it.
//
// Rows.  The query heads of one key/value head see the same keys, so a row is
// a (token, query head) pair, r = token * group + head: a tile of rows reads
// each key once for all of them, and a decode step's single token still fills
// `group` columns of a matrix instruction.
//
// Products.  Both are transposed: S' = K Q' has one query row to a column, so
// a lane holds several keys' scores of one row; their maximum needs one or two
// exchanges between lanes, and the weights are already where the second
// product, O' = V' P', takes its right operand, up to an order of the keys
// that V' is read in as well.  V' comes out of row-major shared memory through
// the transposing read (ds_read_b64_tr_b16: of a 4 x 16 block whose row i is
// given by lanes 4 i .. 4 i + 3 of sixteen, lane j gets column j).
//
// c > 0: the sign of a negative scale goes into q, and a scale of 0 is a q of 0.
//
// What a row does not see is not read, or its score is set to -infinity; a
// value row that some rows of a tile see and others do not is multiplied by an
// exact 0 for the latter, except that 0 * infinity is NaN: where tiles lie on the
// mask's edge, such values are taken out on their way to shared memory, and a
// loop adds them to the rows that see them (`add_special`).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "cache_internal.h"
#include "cache_types.h"

namespace kvc {
namespace {

constexpr float kSlack = 8.0f;
template <class V>   // the type that weights are rounded to
constexpr float kLift = __is_same(V, Fp16) ? 7.0f : 0.0f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kSingleWaves = 4;   // of the kernel for few rows: each its own keys
constexpr int kSingleRows = 16;
constexpr int kMaxRowBytes = KVCACHE_MAX_ATTENTION_HEAD_DIM * 2;

typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// A format's rows as the matrix instructions take them.  V: the type of the
// second product.  8-bit codes become bf16 there whatever the queries' type,
// since a weight times a value's scale may leave fp16's range.
template <class T, class F>
struct Held {
    static constexpr bool coded = true;
    static constexpr int kShift = 3;   // log2 of a piece's bytes
    typedef u32x2 piece;   // 8 codes
    typedef Bf16 V;
    static __device__ __forceinline__ u32x4 key(piece p) { return Widen<T, F>::eight(p); }
    static __device__ __forceinline__ u32x4 value(piece p) { return Widen<Bf16, F>::eight(p); }
    // four values as two words of V
    static __device__ __forceinline__ u32x2 value4(const uint8_t *p)
    {
        const u32x4 w = Widen<Bf16, F>::eight(u32x2{*(const uint32_t *)p, 0});
        return u32x2{w.x, w.y};
    }
};
template <class T>
struct Held<T, void> {
    static constexpr bool coded = false;
    static constexpr int kShift = 4;
    typedef u32x4 piece;   // 8 values
    typedef T V;
    static __device__ __forceinline__ u32x4 key(piece p) { return p; }
    static __device__ __forceinline__ u32x4 value(piece p) { return p; }
    static __device__ __forceinline__ u32x2 value4(const uint8_t *p) { return *(const u32x2 *)p; }
};

// Lanes 0-31 and 32-63 exchange.
__device__ __forceinline__ float other_half(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float((threadIdx.x & 32u) ? r[0] : r[1]);
}

// Eight values of one column, keys `first` .. + 3 and `second` .. + 3 of the
// lane's group of sixteen, from row-major shared memory: `at` is this lane's
// address for row first + (lane % 16) / 4 and columns 4 (lane % 4) .. + 3.
__device__ __forceinline__ u32x4 columns(const uint8_t *at, int second)
{
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)at));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + second)));
    return u32x4{a.x, a.y, b.x, b.y};
}

// Where reads of shared memory and products stay on their side (vector and
// scalar arithmetic may pass).  Left alone, the compiler sinks each read to
// its product and waits there.
__device__ __forceinline__ void keep_order()
{
    __builtin_amdgcn_sched_barrier(0x2 | 0x4 | 0x400);
}

// N products in order, the operands of each read four products ahead: read(n)
// gives product n's, use(n, operand) takes it.  The first four may come from
// an earlier `begin`.
template <class E, int N>
struct Feed {
    E f[2][4];
    template <class Read>
    __device__ __forceinline__ void begin(Read &&read)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[0][i] = read(i);
        keep_order();
    }
    template <class Read, class Use>
    __device__ __forceinline__ void run(Read &&read, Use &&use)
    {
#pragma unroll
        for (int g = 0; g < N / 4; ++g) {
            if (g + 1 < N / 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[(g + 1) & 1][i] = read(4 * (g + 1) + i);
            }
            keep_order();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                use(4 * g + i, f[g & 1][i]);
            keep_order();
        }
    }
};

// Takes infinities and NaN out of eight 16-bit values; whether there were any.
template <class T>
__device__ __forceinline__ bool clean(u32x4 &p)
{
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool lo = (p[i] & T::kExponent) == T::kExponent;
        const bool hi = (p[i] >> 16 & T::kExponent) == T::kExponent;
        p[i] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
        any |= lo || hi;
    }
    return any;
}

// Whether there are any in N times eight: without their signs, 16-bit floats
// order like their bits.
template <class T, int N>
__device__ __forceinline__ bool any_special(const u32x4 *p)
{
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            most = max_halves(most, p[i][j] & 0x7fff7fffu);
    return (most & 0xffffu) >= T::kExponent || most >> 16 >= T::kExponent;
}

// Adds the infinities and NaN among four values of a row that is seen.
template <class H>
__device__ __forceinline__ void add_special(const uint8_t *at, bool sees, float *o)
{
    const u32x2 w = H::value4(at);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = (float)__builtin_bit_cast(typename H::V::elem, (uint16_t)(w[j / 2] >> (16 * (j % 2))));
        o[j] += sees && !__builtin_isfinite(x) ? x : 0.0f;
    }
}

// The sequence of this workgroup: its query rows and keys, bounded by what the
// host said, so that no value in q_starts or context_lens leads outside.
struct Sequence {
    int32_t q0, n, ctx, bound;   // first token, tokens, context, tokens that may be looked up
};
__device__ __forceinline__ Sequence sequence_of(const AttentionArgs &a, uint32_t s)
{
    Sequence r;
    const int32_t first = a.q_starts[s], end = a.q_starts[s + 1], total = (int32_t)a.total_q;
    r.q0 = first < 0 ? 0 : first < total ? first : total;
    const int32_t q1 = end < r.q0 ? r.q0 : end < total ? end : total;
    r.n = q1 - r.q0;
    r.ctx = a.context_lens[s];
    bool bad = first != r.q0 || end != q1 || r.ctx < 0;
    if (r.ctx < 0)
        r.ctx = 0;
    r.bound = r.ctx < (int32_t)a.max_context ? r.ctx : (int32_t)a.max_context;
    bad |= r.ctx != r.bound;
    if (r.n > (int32_t)a.max_q_len)
        bad = true;
    if (bad && threadIdx.x == 0)
        set_status(a.status, KVCACHE_BAD_LENGTH);
    return r;
}

// Where rows that read as zeros are read: those past a sequence's keys, and of
// page numbers out of range.  (An address picked costs less than a branch
// around each read.)
static __device__ const u32x4 kZeros[kMaxRowBytes / 16] = {};

// What the table says for token t, or for the last one from `end` > 0 on.
// Looked up ahead, and checked (checked_page) where it is used: a check beside
// the load would wait for it, and for every load before it.
__device__ __forceinline__ uint32_t raw_page(const AttentionArgs &a, const int32_t *table, int32_t t, int32_t end)
{
    return (uint32_t)table[a.page_size.div((uint32_t)(t < end ? t : end - 1))];
}

// The page of token t < end; ~0 from `end` on, and for a number out of range.
__device__ __forceinline__ uint32_t checked_page(const AttentionArgs &a, uint32_t raw, int32_t t, int32_t end)
{
    if (t < end && raw >= a.num_pages)
        set_status(a.status, KVCACHE_BAD_PAGE);
    return t < end && raw < a.num_pages ? raw : ~0u;
}

// The address of token t's row: strides in units of 2^Shift bytes, which 32
// bits hold (a product of 64-bit strides takes three times the instructions).
template <int Shift>
__device__ __forceinline__ uint64_t row_address(const AttentionArgs &a, uint32_t page, int32_t t, const void *base,
                                                uint32_t page_stride, uint32_t place_stride)
{
    const uint32_t place = a.page_size.mod((uint32_t)t, a.page_size.div((uint32_t)t));
    uint64_t at = (uint64_t)base + (((uint64_t)(page == ~0u ? 0 : page) * page_stride +
                                     (uint64_t)place * place_stride) << Shift);
    asm volatile("" : "+v"(at));   // picked below, not branched around
    return page == ~0u ? (uint64_t)kZeros : at;
}

// A piece at an address that came out of shared memory: global, not flat.
template <class P>
__device__ __forceinline__ P load_at(uint64_t address)
{
    return *(const __attribute__((address_space(1))) P *)address;
}

// The same past the caches.
template <class P>
__device__ __forceinline__ P load_once_at(uint64_t address)
{
    return __builtin_nontemporal_load((const __attribute__((address_space(1))) P *)address);
}

// Four results of a row, as consecutive 16-bit values.
template <class T>
__device__ __forceinline__ void store4(typename T::elem *out, const float *x)
{
    u32x2 w;
    w.x = pack2<T>(x[0], x[1]);
    w.y = pack2<T>(x[2], x[3]);
    *(u32x2 *)out = w;
}

// ---- many rows --------------------------------------------------------------
//
// A workgroup of kWaves wavefronts takes 32 * kWaves rows of one (sequence,
// key/value head) and walks the keys in tiles of kKeys, all wavefronts reading
// the same tile from shared memory.  A wavefront's work on tile i is a block of
// matrix products, O += V(i-1) P(i-1) and S = K(i) Q, and a block of vector
// arithmetic, the softmax of S; with two wavefronts on a SIMD, one does its
// products while the other does its softmax: the workgroup's two halves run the
// same loop, one barrier apart (a "phase" is what lies between two barriers;
// the first half does products in even phases, the second in odd ones).
//
//   phase     first half                           second half
//   2 i       outputs(i - 1), scores(i)            stage(i), softmax(i - 1)
//   2 i + 1   stage(i), softmax(i)                 outputs(i - 1), scores(i)
//
// stage(i) moves a thread's share of K(i + 1) and V(i) from registers into
// shared memory and sends for that of K(i + 2) and V(i + 1).  K(i) and V(i - 1)
// are read in phases 2 i and 2 i + 1 and their successors in the same buffers
// are written in 2 i + 2 at the earliest, so two buffers do.
// Addresses of the rows come from a table in shared memory, written by one lane
// for each key four tiles ahead (worked out by every thread for its own pieces
// they took more vector instructions than the softmax).
//
// Rows of shared memory are padded so that neither the 16-byte reads of K
// (stride = 16 bytes mod 256) nor the transposing reads of V (64 mod 256) meet
// in a bank (SQ_LDS_BANK_CONFLICT is 0).
//
// Weights go into the second product rounded once, to 8 bits in bf16 and 11 in
// fp16, and their sum unrounded: over many keys the roundings cancel, and the
// result's relative error is 0.0023 in bf16 where its own rounding alone gives
// 0.0017 (0.00029 and 0.00021 in fp16).  A second part as in the kernel for few
// rows is half the products again: 828 us for the chunk below.
//
// A chunk of 2048 tokens over 18,432, 32 + 8 heads of 128, bf16: 600 us, 970
// TFLOP/s, where a large bf16 product reaches 1,340.  Bound by the products'
// phase: of its 2,200 cycles 1,024 are products, the rest the first operands'
// way from shared memory, the barriers, and the clock that the matrix units
// leave (2.0 to 2.1 GHz); a copy without the second product takes 454 us, one
// without the exponentials 568.  One workgroup of 8 wavefronts to a CU took
// the place of two of 4, whose phases fell as they came (689 us).

template <int DP>
struct TileShape {
    // O and Q of head dimension 256 leave no room for a second wavefront on a SIMD
    static constexpr int kWaves = DP <= 128 ? 8 : 4;
    static constexpr bool kHalves = kWaves == 8;
    static constexpr int kRows = 32 * kWaves;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kKeys = DP <= 128 ? 64 : 32;
    static constexpr int kKStride = DP * 2 + 16;
    static constexpr int kVStride = DP * 2 + 64;
    static constexpr int kKBytes = kKeys * kKStride;
    static constexpr int kVBytes = kKeys * kVStride;
    static constexpr int kPieces = DP / 8;                                // of a row
    static constexpr int kRowsAtOnce = kThreads / kPieces;
    static constexpr int kPasses = kKeys / kRowsAtOnce;
    static constexpr int kRing = 4;                                       // tiles a table or scales are kept for
};

// All wavefronts' shared memory accesses before it come before those after it.
__device__ __forceinline__ void local_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Full: head_dim is DP, and no piece lies behind a row's end.
template <class T, class F, int DP, bool Full>
__global__ __launch_bounds__(TileShape<DP>::kThreads, TileShape<DP>::kHalves ? 2 : 1) void
kvcache_attention_tile_kernel(const AttentionArgs a)
{
    typedef TileShape<DP> S;
    typedef Held<T, F> H;
    typedef typename H::V V;
    typedef typename H::piece Piece;
    // fp16 results of 8-bit pages, whose second product takes bf16: each weight
    // as its rounding and the rest, or the results would keep 8 bits, not 11
    constexpr bool kTwice = H::coded && __is_same(T, Fp16);
    __shared__ __align__(16) uint8_t k_lds[2][S::kKBytes];
    __shared__ __align__(16) uint8_t v_lds[2][S::kVBytes];
    __shared__ uint64_t k_table[S::kRing][S::kKeys], v_table[S::kRing][S::kKeys];
    __shared__ __align__(16) float k_scales[S::kRing][S::kKeys], v_scales[S::kRing][S::kKeys];
    __shared__ uint32_t special[2 * S::kRing];   // whether V(i) has infinities or NaN; twice the ring: read late

    const uint32_t tid = threadIdx.x, lane = tid & 63u, half = lane >> 5, col = lane & 31u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool second = S::kHalves && wave >= S::kWaves / 2;
    // key/value heads fastest: workgroups next to each other go to different
    // XCDs, so the tiles of one head, which read the same keys, share an L2;
    // the last tiles, with the most keys, come first
    uint32_t x = blockIdx.x;
    const uint32_t head = x % a.kv_heads;
    x /= a.kv_heads;
    const uint32_t split = x % a.splits;
    const uint32_t tile = a.tiles - 1 - x / a.splits;
    const Sequence seq = sequence_of(a, blockIdx.y);
    const int32_t *table = a.table + blockIdx.y * a.table_stride;

    const uint32_t rows = (uint32_t)seq.n * a.group.d;
    const uint32_t row0 = tile * S::kRows;
    if (row0 >= rows)
        return;
    const uint32_t row_last = (row0 + S::kRows < rows ? row0 + S::kRows : rows) - 1;
    const int32_t shift = seq.ctx - seq.n;
    const int32_t first = shift + (int32_t)a.group.div(row0), last = shift + (int32_t)a.group.div(row_last);
    const KeyRange seen = key_range(first, last, a.window, seq.bound);
    const KeyRange part = split_range(seen, a.window > 0 ? seen.lo : 0, split, a.split_keys);
    const int32_t lo = part.lo, hi = part.hi;

    // this lane's row
    const uint32_t row = row0 + wave * 32 + col;
    const bool held = row < rows;
    const uint32_t token = a.group.div(held ? row : 0), member = a.group.mod(held ? row : 0, token);
    const int32_t pos = shift + (int32_t)token;
    const int32_t see_hi = held ? (pos < hi - 1 ? pos : hi - 1) : -1;                 // last key seen
    const int32_t see_lo = first_seen(pos, a.window);
    // a row sees key t if t - see_lo is below see_count, unsigned
    const uint32_t see_count = see_hi < see_lo ? 0 : (uint32_t)(see_hi - see_lo) + 1;

    f32x16 o[DP / 32] = {};
    float m = -__builtin_inff(), l = 0.0f;

    if (lo < hi) {
        typename T::eight q[DP / 16];
        {
            const typename T::elem *at = (const typename T::elem *)a.q + (int64_t)(seq.q0 + token) * a.q_st +
                                         (int64_t)(head * a.group.d + member) * a.q_sh;
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const uint32_t d = s * 16 + half * 8;
                u32x4 p = {};
                if (held && (Full || d < a.head_dim))
                    p = (*(const u32x4 *)(at + d) & a.q_keep) ^ a.q_flip;
                q[s] = __builtin_bit_cast(typename T::eight, p);
            }
        }
        const int32_t tiles = (hi - lo + S::kKeys - 1) / S::kKeys;
        const uint32_t esize = H::coded ? 1 : 2;
        const uint8_t *k_base = (const uint8_t *)a.k + (int64_t)head * a.k_head * esize;
        const uint8_t *v_base = (const uint8_t *)a.v + (int64_t)head * a.v_head * esize;
        const float *ks_base = a.k_scale + (int64_t)head * a.ks_head, *vs_base = a.v_scale + (int64_t)head * a.vs_head;

        // ---- tables and scales: wavefronts 0 and 1 write rows' addresses,
        // 2 and 3 an 8-bit format's scales, a lane for each key
        uint32_t raw = 0;       // what the page table says, looked up a tile ahead
        float scale = 0.0f;
        const auto look_up = [&](int32_t i) { raw = raw_page(a, table, lo + i * S::kKeys + (int32_t)lane, hi); };
        const auto write_table = [&](int32_t i) {   // of tile i; raw is its
            const int32_t t = lo + i * S::kKeys + (int32_t)lane;
            const uint32_t page = checked_page(a, raw, t, hi);
            if (wave == 0) {
                if (lane < S::kKeys)
                    k_table[i & (S::kRing - 1)][lane] = row_address<H::kShift>(a, page, t, k_base, a.k_page, a.k_place);
                if (lane == 0)
                    special[i & (2 * S::kRing - 1)] = 0;
            } else if (lane < S::kKeys) {
                v_table[i & (S::kRing - 1)][lane] = row_address<H::kShift>(a, page, t, v_base, a.v_page, a.v_place);
            }
        };
        const auto load_scale = [&](int32_t i) {
            const int32_t t = lo + i * S::kKeys + (int32_t)lane;
            const uint32_t page = checked_page(a, raw, t, hi);
            scale = load_at<float>(wave == 2 ? row_address<2>(a, page, t, ks_base, a.ks_page, a.ks_place)
                                             : row_address<2>(a, page, t, vs_base, a.vs_page, a.vs_place));
        };
        const auto write_scale = [&](int32_t i) {
            if (lane < S::kKeys)
                (wave == 2 ? k_scales : v_scales)[i & (S::kRing - 1)][lane] = scale;
        };
        // what goes with outputs(i) in these wavefronts
        const auto ahead = [&](int32_t i) {
            if (wave < 2) {
                write_table(i + 4);
                look_up(i + 5);
            } else if (H::coded && wave < 4) {
                write_scale(i + 1);
                load_scale(i + 2);
                look_up(i + 3);
            }
        };

        // ---- a thread's share of the rows: piece tid % kPieces of keys
        // tid / kPieces + j * kRowsAtOnce
        const uint32_t piece = tid % S::kPieces, key0 = tid / S::kPieces;
        const bool in = Full || piece * 8 < a.head_dim;
        Piece k_next[S::kPasses], v_next[S::kPasses];
        uint64_t k_from[S::kPasses], v_from[S::kPasses];   // of the rows sent for next
        const auto find = [&](int32_t i) {
#pragma unroll
            for (int j = 0; j < S::kPasses; ++j) {
                k_from[j] = k_table[(i + 2) & (S::kRing - 1)][key0 + j * S::kRowsAtOnce];
                v_from[j] = v_table[(i + 1) & (S::kRing - 1)][key0 + j * S::kRowsAtOnce];
            }
        };
        const auto load = [&](Piece *next, const uint64_t *from) {
#pragma unroll
            for (int j = 0; j < S::kPasses; ++j)
                next[j] = load_at<Piece>(in ? from[j] + piece * 8 * esize : (uint64_t)kZeros);
        };
        // not every row sees every key of the tile
        const auto on_edge = [&](int32_t i) {
            const int32_t t0 = lo + i * S::kKeys;
            return t0 + S::kKeys - 1 > first || t0 + S::kKeys > hi || (a.window > 0 && t0 <= last - a.window);
        };
        const auto put_keys = [&](int32_t i) {
#pragma unroll
            for (int j = 0; j < S::kPasses; ++j)
                *(u32x4 *)(k_lds[i & 1] + (key0 + j * S::kRowsAtOnce) * S::kKStride + piece * 16) = H::key(k_next[j]);
        };
        const auto put_values = [&](int32_t i) {
            const bool edge = on_edge(i);
            bool any = false;
#pragma unroll
            for (int j = 0; j < S::kPasses; ++j) {
                u32x4 w = H::value(v_next[j]);
                if (edge)
                    any |= clean<V>(w);
                *(u32x4 *)(v_lds[i & 1] + (key0 + j * S::kRowsAtOnce) * S::kVStride + piece * 16) = w;
            }
            if (edge && any)
                special[i & (2 * S::kRing - 1)] = 1;
        };
        // Nothing here is conditional on i: what lies behind the last tile reads
        // as zeros, and a load that may or may not follow another makes a wait
        // for either a wait for both.
        const auto put = [&](int32_t i) {
            put_keys(i + 1);
            put_values(i);
        };
        const auto send = [&] {
            load(k_next, k_from);
            load(v_next, v_from);
        };

        // ---- the first tables, scales and rows, each kind of read sent at once
        if (wave < 2) {
            uint32_t ahead_raw[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                look_up(i);
                ahead_raw[i] = raw;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                raw = ahead_raw[i];
                write_table(i);
            }
            raw = ahead_raw[4];
        } else if (H::coded && wave < 4) {
            uint32_t ahead_raw[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                look_up(i);
                ahead_raw[i] = raw;
            }
            raw = ahead_raw[0];
            load_scale(0);
            const float scale_0 = scale;
            raw = ahead_raw[1];
            load_scale(1);
            const float scale_1 = scale;
            scale = scale_0;
            write_scale(0);
            scale = scale_1;
            raw = ahead_raw[2];
        }
        local_barrier();
        {
            Piece k_first[S::kPasses];
            find(-2);
            load(k_first, k_from);
            find(-1);
            send();
#pragma unroll
            for (int j = 0; j < S::kPasses; ++j)
                *(u32x4 *)(k_lds[0] + (key0 + j * S::kRowsAtOnce) * S::kKStride + piece * 16) = H::key(k_first[j]);
        }
        if (second) {
            put(0);
            find(0);
            send();
        }
        find(second ? 1 : 0);
        local_barrier();

        // ---- the two blocks of work
        f32x16 s[S::kKeys / 32];
        typename V::eight p[S::kKeys / 16], rest[kTwice ? S::kKeys / 16 : 1];
        constexpr int kBlocks = S::kKeys / 32;
        const uint32_t k_lane = col * S::kKStride + half * 16;
        // of a block of 16 keys, keys 4 half .. + 3 and 8 + 4 half .. + 3
        const uint32_t v_lane = (half * 4 + (lane % 16) / 4) * S::kVStride + ((lane / 16) % 2) * 32 + (lane % 4) * 8;

        const auto read_k = [&](int32_t i, int n) {
            return *(const typename T::eight *)(k_lds[i & 1] + k_lane + n % kBlocks * 32 * S::kKStride + n / kBlocks * 32);
        };
        const auto read_v = [&](int32_t i, int n) {
            return __builtin_bit_cast(typename V::eight,
                                      columns(v_lds[i & 1] + v_lane + n / (DP / 32) * 16 * S::kVStride +
                                              n % (DP / 32) * 64, 8 * S::kVStride));
        };
        Feed<typename T::eight, kBlocks * DP / 16> k_feed;
        // K's first reads go out ahead of the outputs where registers are left
        constexpr bool kEarly = DP <= 128 && Full && !H::coded;
        const auto scores = [&](int32_t i) {
            if (!kEarly)
                k_feed.begin([&](int n) { return read_k(i, n); });
            k_feed.run([&](int n) { return read_k(i, n); }, [&](int n, typename T::eight k) {
                const int b = n % kBlocks, d = n / kBlocks;
                s[b] = T::mfma32(k, q[d], d == 0 ? f32x16{} : s[b]);
            });
        };
        const auto outputs = [&](int32_t i) {
            Feed<typename V::eight, S::kKeys / 16 * DP / 32> feed;
            feed.begin([&](int n) { return read_v(i, n); });
            if (kEarly)
                k_feed.begin([&](int n) { return read_k(i + 1, n); });
            ahead(i);
            find(second ? i + 2 : i + 1);
            feed.run([&](int n) { return read_v(i, n); }, [&](int n, typename V::eight v) {
                o[n % (DP / 32)] = V::mfma32(v, p[n / (DP / 32)], o[n % (DP / 32)]);
                if constexpr (kTwice)
                    o[n % (DP / 32)] = V::mfma32(v, rest[n / (DP / 32)], o[n % (DP / 32)]);
            });
            if (on_edge(i) && __builtin_amdgcn_readfirstlane(special[i & (2 * S::kRing - 1)])) {
                const int32_t t0 = lo + i * S::kKeys;
#pragma unroll 1
                for (int32_t t = t0; t < t0 + S::kKeys && t < hi; ++t) {
                    const uint32_t from = checked_page(a, raw_page(a, table, t, hi), t, hi);
                    if (from == ~0u)
                        continue;
                    const bool sees = (uint32_t)(t - see_lo) < see_count;
                    const uint8_t *at_v = (const uint8_t *)row_address<H::kShift>(a, from, t, v_base, a.v_page, a.v_place) +
                                          half * 4 * esize;
#pragma unroll
                    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float y[4] = {};
                            if (Full || d * 32 + j * 8 + half * 4 < a.head_dim)
                                add_special<H>(at_v + (d * 32 + j * 8) * esize, sees, y);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[d][4 * j + e] += y[e];
                            __builtin_amdgcn_sched_barrier(0);
                        }
                }
            }
        };
        const auto softmax = [&](int32_t i) {
            // register 4 j + e of block b is key t0 + 32 b + 8 j + 4 half + e
            const float *ks = k_scales[i & (S::kRing - 1)] + half * 4, *vs = v_scales[i & (S::kRing - 1)] + half * 4;
            if (H::coded) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 c = *(const f32x4 *)(ks + b * 32 + j * 8);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[b][4 * j + e] *= c[e];
                    }
            }
            if (on_edge(i)) {
                const uint32_t see = (uint32_t)(lo + i * S::kKeys + (int32_t)half * 4 - see_lo);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        s[b][j] = see + (b * 32 + (j / 4) * 8 + j % 4) < see_count ? s[b][j] : -__builtin_inff();
            }
            // the running maximum, in units of log2
            float top = s[0][0];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    top = __builtin_fmaxf(top, s[b][j]);
            top = __builtin_fmaxf(top, other_half(top)) * a.scale_log2;
            if (__builtin_amdgcn_ballot_w64(top > m + (kLift<V> + kSlack))) {
                const float grown = __builtin_fmaxf(m, top - kLift<V>);
                const float shrink = m == grown ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
                m = grown;
                l *= shrink;
#pragma unroll
                for (int d = 0; d < DP / 32; ++d)
                    o[d] *= shrink;
            }
            const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                float w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][j], a.scale_log2, -base));
                    l += w[j];
                }
                if (H::coded) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 c = *(const f32x4 *)(vs + b * 32 + j * 8);
                        // a hidden row's scale may be anything
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[4 * j + e] = s[b][4 * j + e] == -__builtin_inff() ? 0.0f : w[4 * j + e] * c[e];
                    }
                }
                p[2 * b] = __builtin_bit_cast(typename V::eight, pack8<V>(w));
                p[2 * b + 1] = __builtin_bit_cast(typename V::eight, pack8<V>(w + 8));
                if constexpr (kTwice) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[j] = __builtin_isfinite(w[j]) ? w[j] - (float)p[2 * b + j / 8][j % 8] : 0.0f;
                    rest[2 * b] = __builtin_bit_cast(typename V::eight, pack8<V>(w));
                    rest[2 * b + 1] = __builtin_bit_cast(typename V::eight, pack8<V>(w + 8));
                }
            }
        };

        // No condition around the products: where O may or may not have changed
        // it is copied.  (The scores behind the last tile are of zeros.)
        if (second)
            local_barrier();
        if (kEarly)
            k_feed.begin([&](int n) { return read_k(0, n); });
        scores(0);
        __builtin_amdgcn_sched_barrier(0);
        local_barrier();
        for (int32_t i = 0; i < tiles; ++i) {
            put(second ? i + 1 : i);
            send();
            softmax(i);
            __builtin_amdgcn_sched_barrier(0);
            local_barrier();
            __builtin_amdgcn_s_setprio(1);   // products before the other half's arithmetic: 1%
            outputs(i);
            scores(i + 1);
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            local_barrier();
        }
        if (S::kHalves && !second)
            local_barrier();
    }

    l += other_half(l);
    if (!held)
        return;
    const uint32_t qhead = head * a.group.d + member;
    const int64_t qtoken = seq.q0 + token;
    if (a.splits > 1) {
        const int64_t part = ((int64_t)split * a.total_q + qtoken) * a.q_heads + qhead;
        if (half == 0) {
            a.part_ml[2 * part] = m;
            a.part_ml[2 * part + 1] = l;
        }
        float *to = a.part_o + part * a.head_dim;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at_d = d * 32 + j * 8 + half * 4;
                if ((Full || at_d < a.head_dim) && l != 0.0f)   // else not read
                    *(f32x4 *)(to + at_d) = f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
            }
        return;
    }
    if (a.lse && half == 0)
        a.lse[qtoken * a.l_st + qhead * a.l_sh] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    typename T::elem *to = (typename T::elem *)a.out + qtoken * a.o_st + qhead * a.o_sh;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t at_d = d * 32 + j * 8 + half * 4;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = o[d][4 * j + e] * inv;
            if (Full || at_d < a.head_dim)
                store4<T>(to + at_d, y);
        }
}

// ---- few rows ---------------------------------------------------------------
//
// At most 16 rows a (sequence, key/value head), as in a decode step: bound by
// reading the cache, so everything serves to keep reads in flight.  The keys
// of a split are dealt to the 4 wavefronts of a workgroup in steps of kKeys
// (about 16 KiB of K and V); each keeps its own maximum, sum and output, joined
// at the end.  A wavefront takes K straight from memory into the matrix
// instruction's registers, V through registers into shared memory of its own
// (for the transposing read), and issues the next step's reads as soon as a
// step's registers are free; their addresses were put into shared memory two
// steps ahead, one row a lane.  Nothing is read twice, and V, whose lines a
// read takes whole, passes the caches by (64 x 8192 bf16: 269 us against 286);
// a line of K is split over two to four reads and needs them (302 us).
//
// Of the reads' own rate (6.0 TB/s for scattered blocks) 64 x 8192 in bf16
// reaches 96%, 12 x 40001 in e4m3 86%: there the lookups of lines weigh more,
// two for each half-read line of K, and the joining of the splits (5 us).
//
// The second product has time to spare: a weight goes in as its rounding and
// the rest (two products), so the weights keep 16 bits in bf16 and 22 in fp16.
// A rest of 0 or of the other sign would turn an infinite value into NaN, so
// these are taken out here wherever they are.

template <class H, int DP>
struct SingleShape {
    static constexpr int kKeys = DP == 64 || (DP == 128 && H::coded) ? 64 : 32;
    static constexpr int kVStride = DP * 2 + 32;   // 32 mod 256: see above, for blocks of 16 rows
    static constexpr int kVBytes = kKeys * kVStride;
    static constexpr int kWaveBytes = kVBytes + kKeys * (8 + 16);   // and the scales and addresses
    static constexpr int kBlocks = kKeys / 16;     // of the first product
    static constexpr int kPairs = kKeys / 32;      // and of the second
    static constexpr int kJoinBytes = kSingleWaves * kSingleRows * (DP + 4) * 4;
    static constexpr int kBytes = kSingleWaves * kWaveBytes > kJoinBytes ? kSingleWaves * kWaveBytes : kJoinBytes;
};

// Full: head_dim is DP, so no piece lies behind a row's end, and 8-bit rows can
// be read 16 codes to a lane: of a row's 64 codes, one read takes all, where
// two reads of 8 codes a lane look the same line up twice.
template <class T, class F, int DP, bool Full>
__global__ __launch_bounds__(64 * kSingleWaves, DP == 256 && (__is_same(F, void) || !Full) ? 1 : 2) void kvcache_attention_single_kernel(const AttentionArgs a)
{
    typedef Held<T, F> H;
    typedef SingleShape<H, DP> S;
    typedef typename H::V V;
    constexpr bool kWide = Full && H::coded;
    constexpr int kPieceEights = kWide ? 2 : 1;
    typedef std::conditional_t<kWide, u32x4, typename H::piece> Piece;
    constexpr int kPieces = DP / (8 * kPieceEights);   // of a row
    constexpr int kRowsAtOnce = 64 / kPieces, kPasses = S::kKeys / kRowsAtOnce;
    __shared__ __align__(16) uint8_t lds[S::kBytes];
    __shared__ float join_m[kSingleWaves][kSingleRows], join_l[kSingleWaves][kSingleRows];

    const uint32_t tid = threadIdx.x, lane = tid & 63u, group = lane >> 4, col = lane & 15u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t head = blockIdx.x % a.kv_heads, split = blockIdx.x / a.kv_heads;
    const int32_t *table = a.table + blockIdx.y * a.table_stride;
    // Without a window a split starts where it starts: its first lookup need
    // not wait for the sequence's length (what it gives is checked later).
    const int32_t mine = (int32_t)(lane % S::kKeys);   // the key of a step whose row this lane looks up
    uint32_t raw = 0, raw_1 = 0, raw_2 = 0;
    if (a.window == 0 && a.max_context > 0) {
        const int32_t t = (int32_t)(split * a.split_keys + wave * S::kKeys) + mine;
        raw = raw_page(a, table, t, (int32_t)a.max_context);
        raw_1 = raw_page(a, table, t + S::kKeys * kSingleWaves, (int32_t)a.max_context);
        raw_2 = raw_page(a, table, t + 2 * S::kKeys * kSingleWaves, (int32_t)a.max_context);
    }
    const Sequence seq = sequence_of(a, blockIdx.y);
    uint32_t rows = (uint32_t)seq.n * a.group.d;
    rows = rows < kSingleRows ? rows : kSingleRows;   // more: flagged by sequence_of
    if (rows == 0)
        return;
    const int32_t shift = seq.ctx - seq.n;
    const int32_t first = shift, last = shift + (int32_t)a.group.div(rows - 1);
    const KeyRange seen = key_range(first, last, a.window, seq.bound);
    const KeyRange part = split_range(seen, a.window > 0 ? seen.lo : 0, split, a.split_keys);
    const int32_t lo = part.lo, hi = part.hi;

    const bool held = col < rows;
    const uint32_t token = a.group.div(held ? col : 0), member = a.group.mod(held ? col : 0, token);
    const int32_t pos = shift + (int32_t)token;
    const int32_t see_hi = held ? (pos < hi - 1 ? pos : hi - 1) : -1;
    const int32_t see_lo = first_seen(pos, a.window);
    // a row sees key t if t - see_lo is below see_count, unsigned
    const uint32_t see_count = see_hi < see_lo ? 0 : (uint32_t)(see_hi - see_lo) + 1;

    uint8_t *vlds = lds + wave * S::kWaveBytes;
    float *scales = (float *)(vlds + S::kVBytes);                // of the keys, then of the values
    uint64_t *addresses = (uint64_t *)(scales + 2 * S::kKeys);   // likewise
    f32x4 o[DP / 16] = {};
    float m = -__builtin_inff(), l = 0.0f;

    if (lo < hi) {
        typename T::eight q[DP / 32];
        const typename T::elem *q_at = (const typename T::elem *)a.q + (int64_t)(seq.q0 + token) * a.q_st +
                                       (int64_t)(head * a.group.d + member) * a.q_sh;
#pragma unroll
        for (int s = 0; s < DP / 32; ++s) {
            const uint32_t d = kWide ? s / 2 * 64 + group * 16 + s % 2 * 8 : s * 32 + group * 8;
            u32x4 p = {};
            if (held && (Full || d < a.head_dim))
                p = (*(const u32x4 *)(q_at + d) & a.q_keep) ^ a.q_flip;
            q[s] = __builtin_bit_cast(typename T::eight, p);
        }

        const uint32_t esize = H::coded ? 1 : 2;
        const uint32_t piece = lane % kPieces, vkey = lane / kPieces;
        Piece kp[S::kBlocks][DP / 32 / kPieceEights], vp[kPasses];
        uint64_t k_scale_at, v_scale_at;
        float k_scale = 0.0f, v_scale = 0.0f;
        const uint8_t *k_base = (const uint8_t *)a.k + (int64_t)head * a.k_head * esize;
        const uint8_t *v_base = (const uint8_t *)a.v + (int64_t)head * a.v_head * esize;

        auto look_up = [&](int32_t t0) { raw = raw_page(a, table, t0 + mine, hi); };
        auto put_table = [&](int32_t t0) {
            const int32_t t = t0 + mine;
            const uint32_t page = checked_page(a, raw, t, hi);
            if (S::kKeys == 64 || lane < 32)
                addresses[mine] = row_address<H::kShift>(a, page, t, k_base, a.k_page, a.k_place);
            if (S::kKeys == 64 || lane >= 32)
                addresses[S::kKeys + mine] = row_address<H::kShift>(a, page, t, v_base, a.v_page, a.v_place);
            if (H::coded) {
                k_scale_at = row_address<2>(a, page, t, a.k_scale + (int64_t)head * a.ks_head, a.ks_page, a.ks_place);
                v_scale_at = row_address<2>(a, page, t, a.v_scale + (int64_t)head * a.vs_head, a.vs_page, a.vs_place);
            }
        };
        auto load_rows = [&]() {
            if (H::coded) {
                k_scale = load_at<float>(k_scale_at);
                v_scale = load_at<float>(v_scale_at);
            }
#pragma unroll
            for (int b = 0; b < S::kBlocks; ++b) {
                const uint64_t at = addresses[b * 16 + col] + group * sizeof(Piece);
#pragma unroll
                for (int s = 0; s < DP / 32 / kPieceEights; ++s)
                    kp[b][s] = load_at<Piece>(Full || s * 32 + group * 8 < a.head_dim ? at + s * 4 * sizeof(Piece)
                                                                                     : (uint64_t)kZeros);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const uint64_t at = addresses[S::kKeys + i * kRowsAtOnce + vkey] + piece * sizeof(Piece);
                vp[i] = load_once_at<Piece>(Full || piece * 8 < a.head_dim ? at : (uint64_t)kZeros);
            }
        };

        // Eight of a piece, as the products take them.
        const auto key_of = [&](int b, int i) {
            if constexpr (kWide)
                return H::key(i % 2 ? u32x2{kp[b][i / 2].z, kp[b][i / 2].w} : u32x2{kp[b][i / 2].x, kp[b][i / 2].y});
            else
                return H::key(kp[b][i]);
        };
        const auto value_of = [&](int i, int e) {
            if constexpr (kWide)
                return H::value(e ? u32x2{vp[i].z, vp[i].w} : u32x2{vp[i].x, vp[i].y});
            else
                return H::value(vp[i]);
        };

        // A wavefront's own writes to shared memory are read by other lanes of
        // it: in order in the LDS queue, and kept in order in the code by these
        // fences, which are no instructions.
        const auto in_order = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
        constexpr int kStep = S::kKeys * kSingleWaves;
        int32_t t0 = lo + (int32_t)wave * S::kKeys;
        if (a.window > 0) {
            look_up(t0 + kStep);
            raw_1 = raw;
            look_up(t0 + 2 * kStep);
            raw_2 = raw;
            look_up(t0);
        }
        put_table(t0);
        in_order();
        load_rows();
        in_order();
        raw = raw_1;
        put_table(t0 + kStep);
        raw = raw_2;
        for (; t0 < hi; t0 += kStep) {
            f32x4 s[S::kBlocks] = {};
#pragma unroll
            for (int i = 0; i < DP / 32; ++i)
#pragma unroll
                for (int b = 0; b < S::kBlocks; ++b)
                    s[b] = T::mfma16(__builtin_bit_cast(typename T::eight, key_of(b, i)), q[i], s[b]);
            if (H::coded) {
                scales[mine] = k_scale;
                scales[S::kKeys + mine] = v_scale;
            }
            // not every row sees every key
            const bool edge = t0 + S::kKeys - 1 > first || t0 + S::kKeys > hi ||
                              (a.window > 0 && t0 <= last - a.window);
            bool special = false;
            constexpr int kEights = kPasses * kPieceEights;
            u32x4 values[kEights];
#pragma unroll
            for (int i = 0; i < kEights; ++i)
                values[i] = value_of(i / kPieceEights, i % kPieceEights);
            if (!H::coded)
                special = __builtin_amdgcn_ballot_w64(any_special<V, kEights>(values)) != 0;
            if (special || edge) {
                special = false;
#pragma unroll
                for (int i = 0; i < kEights; ++i)
                    special |= clean<V>(values[i]);
                special = __builtin_amdgcn_ballot_w64(special) != 0;
            }
#pragma unroll
            for (int i = 0; i < kEights; ++i)
                *(u32x4 *)(vlds + (i / kPieceEights * kRowsAtOnce + vkey) * S::kVStride +
                           (piece * kPieceEights + i % kPieceEights) * 16) = values[i];
            in_order();
            load_rows();   // of the next step: zeros behind the last key

            // register j of block b is key t0 + 16 b + 4 group + j
            if (H::coded) {
#pragma unroll
                for (int b = 0; b < S::kBlocks; ++b)
                    s[b] *= *(const f32x4 *)(scales + b * 16 + group * 4);
            }
            if (edge) {
                const uint32_t see = (uint32_t)(t0 + (int32_t)group * 4 - see_lo);
#pragma unroll
                for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[b][j] = see + (b * 16 + j) < see_count ? s[b][j] : -__builtin_inff();
            }
            float top = s[0][0];
#pragma unroll
            for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    top = __builtin_fmaxf(top, s[b][j]);
            top = __builtin_fmaxf(top, other_half(top));
            top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64)) * a.scale_log2;
            if (__builtin_amdgcn_ballot_w64(top > m + (kLift<V> + kSlack))) {
                const float grown = __builtin_fmaxf(m, top - kLift<V>);
                const float shrink = m == grown ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
                m = grown;
                l *= shrink;
#pragma unroll
                for (int d = 0; d < DP / 16; ++d)
                    o[d] *= shrink;
            }
            const float base = m == -__builtin_inff() ? 0.0f : m;
            typename V::eight p[S::kPairs], rest[S::kPairs];
#pragma unroll
            for (int i = 0; i < S::kPairs; ++i) {
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + j / 4][j % 4], a.scale_log2, -base));
                    l += w[j];
                }
                if (H::coded) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const f32x4 c = *(const f32x4 *)(scales + S::kKeys + (2 * i + b) * 16 + group * 4);
                        // a hidden row's scale may be anything
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[4 * b + j] = s[2 * i + b][j] == -__builtin_inff() ? 0.0f : w[4 * b + j] * c[j];
                    }
                }
                p[i] = __builtin_bit_cast(typename V::eight, pack8<V>(w));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float r = w[j] - (float)p[i][j];
                    w[j] = __builtin_isfinite(w[j]) ? r : 0.0f;
                }
                rest[i] = __builtin_bit_cast(typename V::eight, pack8<V>(w));
            }

            // keys 4 group .. + 3 and 16 + 4 group .. + 3 of a pair of blocks,
            // columns 16 d + lane % 16
            const uint8_t *vat = vlds + (group * 4 + col / 4) * S::kVStride + (col % 4) * 8;
            const auto read_v = [&](int n) {
                return __builtin_bit_cast(typename V::eight, columns(vat + n / (DP / 16) * 32 * S::kVStride +
                                                                     n % (DP / 16) * 32, 16 * S::kVStride));
            };
            Feed<typename V::eight, S::kPairs * DP / 16> feed;
            feed.begin(read_v);
            feed.run(read_v, [&](int n, typename V::eight v) {
                const int d = n % (DP / 16), i = n / (DP / 16);
                o[d] = V::mfma16(v, p[i], o[d]);
                o[d] = V::mfma16(v, rest[i], o[d]);
            });
            if (special) {
#pragma unroll 1
                for (int32_t t = t0; t < t0 + S::kKeys && t < hi; ++t) {
                    const uint32_t from = checked_page(a, raw_page(a, table, t, hi), t, hi);
                    if (from == ~0u)
                        continue;
                    const bool sees = (uint32_t)(t - see_lo) < see_count;
                    const uint8_t *at_v = (const uint8_t *)row_address<H::kShift>(a, from, t, v_base, a.v_page, a.v_place) +
                                          group * 4 * esize;
#pragma unroll
                    for (int d = 0; d < DP / 16; ++d) {
                        float x[4] = {};
                        if (Full || d * 16 + group * 4 < a.head_dim)
                            add_special<H>(at_v + d * 16 * esize, sees, x);
                        o[d] += f32x4{x[0], x[1], x[2], x[3]};
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            // the next step's writes stay behind these reads
            in_order();
            put_table(t0 + 2 * kStep);
            look_up(t0 + 3 * kStep);
        }
    }

    // join the four wavefronts
    l += other_half(l);
    l += __shfl_xor(l, 16, 64);
    if (lane < 16) {
        join_m[wave][col] = m;
        join_l[wave][col] = l;
    }
    __syncthreads();   // also: every wavefront is done with its V
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kSingleWaves; ++w)
        top = __builtin_fmaxf(top, join_m[w][col]);
    float *joined = (float *)lds;   // [wave][row][DP + 4]
    {
        const float f = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
        float *to = joined + (wave * kSingleRows + col) * (DP + 4);
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
            *(f32x4 *)(to + d * 16 + group * 4) = o[d] * f;
    }
    __syncthreads();
    // a thread takes 4 columns of a row
    for (uint32_t i = tid; i < rows * (DP / 4); i += 64 * kSingleWaves) {
        const uint32_t r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (!Full && d >= a.head_dim)
            continue;
        f32x4 y = {};
        float row_top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kSingleWaves; ++w) {
            y += *(const f32x4 *)(joined + (w * kSingleRows + r) * (DP + 4) + d);
            row_top = __builtin_fmaxf(row_top, join_m[w][r]);
        }
#pragma unroll
        for (int w = 0; w < kSingleWaves; ++w)
            sum += join_m[w][r] == row_top ? join_l[w][r]
                                           : join_l[w][r] * __builtin_amdgcn_exp2f(join_m[w][r] - row_top);
        const uint32_t tok = a.group.div(r), qhead = head * a.group.d + a.group.mod(r, tok);
        const int64_t qtoken = seq.q0 + tok;
        if (a.splits > 1) {
            const int64_t part = ((int64_t)split * a.total_q + qtoken) * a.q_heads + qhead;
            if (d == 0) {
                a.part_ml[2 * part] = row_top;
                a.part_ml[2 * part + 1] = sum;
            }
            if (sum != 0.0f)   // else not read
                *(f32x4 *)(a.part_o + part * a.head_dim + d) = y;
        } else {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float z[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
            store4<T>((typename T::elem *)a.out + qtoken * a.o_st + qhead * a.o_sh + d, z);
            if (a.lse && d == 0)
                a.lse[qtoken * a.l_st + qhead * a.l_sh] =
                    sum == 0.0f ? -__builtin_inff() : (row_top + __builtin_log2f(sum)) * kLn2;
        }
    }
}

// ---- joining splits ---------------------------------------------------------
//
// out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, in a fixed order.  A split
// without keys has l = 0 and is not read.  Over few splits a thread takes 4
// columns of a row and walks them; over more, a workgroup takes a row, its
// threads 4 columns of a split each, as many splits at once as fit, so that the
// reads do not wait for each other (a wavefront that walked 20 splits took
// 13 us; a workgroup a row over 2 splits of 65,536 rows 90 us).

constexpr int kJoinThreads = 256;
constexpr uint32_t kMaxSplits = kJoinThreads;
constexpr uint32_t kFewSplits = 8;

template <class T>
__global__ __launch_bounds__(kJoinThreads) void kvcache_attention_join_few_kernel(const AttentionArgs a)
{
    const uint32_t quads = a.head_dim / 4;
    const uint64_t rows = (uint64_t)a.total_q * a.q_heads;
    const uint64_t row = (uint64_t)blockIdx.x * (kJoinThreads / quads) + threadIdx.x / quads;
    const uint32_t quad = threadIdx.x % quads;
    if (row >= rows || threadIdx.x / quads >= kJoinThreads / quads)
        return;
    f32x2 ml[kFewSplits];
    float m = -__builtin_inff();
#pragma unroll
    for (uint32_t s = 0; s < kFewSplits; ++s) {
        ml[s] = s < a.splits ? *(const f32x2 *)(a.part_ml + 2 * (s * rows + row)) : f32x2{0.0f, 0.0f};
        m = ml[s].y == 0.0f ? m : __builtin_fmaxf(m, ml[s].x);
    }
    float l = 0.0f;
    f32x4 y = {};
#pragma unroll
    for (uint32_t s = 0; s < kFewSplits; ++s) {
        if (ml[s].y != 0.0f) {
            const float w = ml[s].x == m ? 1.0f : __builtin_amdgcn_exp2f(ml[s].x - m);
            l += ml[s].y * w;
            y += *(const f32x4 *)(a.part_o + (s * rows + row) * a.head_dim + quad * 4) * w;
        }
    }
    const int64_t token = row / a.q_heads, head = row % a.q_heads;
    if (a.lse && quad == 0)
        a.lse[token * a.l_st + head * a.l_sh] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float z[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
    store4<T>((typename T::elem *)a.out + token * a.o_st + head * a.o_sh + quad * 4, z);
}

template <class T>
__global__ __launch_bounds__(kJoinThreads) void kvcache_attention_join_kernel(const AttentionArgs a)
{
    __shared__ float weight[kMaxSplits];
    __shared__ float wave_m[kJoinThreads / 64], wave_l[kJoinThreads / 64];
    __shared__ __align__(16) f32x4 part[kJoinThreads];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const int64_t rows = (int64_t)a.total_q * a.q_heads, row = blockIdx.x;

    float m = -__builtin_inff(), l = 0.0f;
    if (tid < a.splits) {
        const f32x2 ml = *(const f32x2 *)(a.part_ml + 2 * (tid * rows + row));
        l = ml.y;
        m = l == 0.0f ? m : ml.x;
    }
    float top = m;
    for (int x = 1; x < 64; x <<= 1)
        top = __builtin_fmaxf(top, __shfl_xor(top, x, 64));
    if (lane == 0)
        wave_m[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 64; ++w)
        top = __builtin_fmaxf(top, wave_m[w]);
    const float f = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
    weight[tid] = l == 0.0f ? -1.0f : f;   // not written
    l = l == 0.0f ? 0.0f : l * f;
    for (int x = 1; x < 64; x <<= 1)
        l += __shfl_xor(l, x, 64);
    if (lane == 0)
        wave_l[wave] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 64; ++w)
        l += wave_l[w];

    const uint32_t quads = a.head_dim / 4, at_once = kJoinThreads / quads;   // head_dim <= 256: 4 at least
    const uint32_t quad = tid % quads, first = tid / quads;
    f32x4 y = {};
    if (first < at_once) {
#pragma unroll 4
        for (uint32_t s = first; s < a.splits; s += at_once) {
            // a weight of 0 counts: it does not hide an infinity or a NaN
            const float w = weight[s];
            if (w >= 0.0f)
                y += *(const f32x4 *)(a.part_o + (s * rows + row) * a.head_dim + quad * 4) * w;
        }
    }
    part[tid] = y;
    __syncthreads();
    if (first != 0)
        return;
    for (uint32_t i = 1; i < at_once; ++i)
        y += part[i * quads + quad];
    const int64_t token = row / a.q_heads, head = row % a.q_heads;
    if (a.lse && quad == 0)
        a.lse[token * a.l_st + head * a.l_sh] = l == 0.0f ? -__builtin_inff() : (top + __builtin_log2f(l)) * kLn2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float z[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
    store4<T>((typename T::elem *)a.out + token * a.o_st + head * a.o_sh + quad * 4, z);
}

template <class T, class F, int DP>
hipError_t attention_pick(const AttentionArgs &a, const AttentionShape &shape, uint32_t num_seqs, hipStream_t s)
{
    const uint32_t blocks = a.kv_heads * a.splits * a.tiles;
    if (shape.single)
        return launch(a.full ? kvcache_attention_single_kernel<T, F, DP, true>
                             : kvcache_attention_single_kernel<T, F, DP, false>,
                      blocks, num_seqs, 64 * kSingleWaves, a, s);
    return launch(a.full ? kvcache_attention_tile_kernel<T, F, DP, true> : kvcache_attention_tile_kernel<T, F, DP, false>,
                  blocks, num_seqs, TileShape<DP>::kThreads, a, s);
}

template <class T, class F>
hipError_t attention_dim(const AttentionArgs &a, const AttentionShape &shape, uint32_t num_seqs, hipStream_t s)
{
    if (a.head_dim <= 64)
        return attention_pick<T, F, 64>(a, shape, num_seqs, s);
    if (a.head_dim <= 128)
        return attention_pick<T, F, 128>(a, shape, num_seqs, s);
    return attention_pick<T, F, 256>(a, shape, num_seqs, s);
}

template <class T>
hipError_t attention_type(const AttentionArgs &a, const AttentionShape &shape, uint32_t num_seqs,
                          uint32_t format, hipStream_t s)
{
    const hipError_t e = format == KVCACHE_FP8    ? attention_dim<T, Fp8>(a, shape, num_seqs, s)
                         : format == KVCACHE_INT8 ? attention_dim<T, Int8>(a, shape, num_seqs, s)
                                                  : attention_dim<T, void>(a, shape, num_seqs, s);
    if (e != hipSuccess || a.splits == 1)
        return e;
    const uint64_t rows = (uint64_t)a.total_q * a.q_heads;
    const uint32_t at_once = kJoinThreads / (a.head_dim / 4);
    if (a.splits <= kFewSplits)
        return launch(kvcache_attention_join_few_kernel<T>, (uint32_t)((rows + at_once - 1) / at_once), 1,
                      kJoinThreads, a, s);
    return launch(kvcache_attention_join_kernel<T>, (uint32_t)rows, 1, kJoinThreads, a, s);
}

}  // namespace

// The layout of a call, from its sizes alone.  Where the rows give fewer
// workgroups than the GPU holds, the keys are split.
//
// Few rows: the GPU holds 512 workgroups, and ragged sequences want several
// times that, of at least 512 keys each (12 x 40001 e4m3, before its values
// passed the caches by: 156 us with at most 1,280 workgroups, 151 with 2,048,
// 157 with 4,096, 173 with 6,144); a call too small for that takes splits of
// one step of a workgroup, for the shortest chain of reads.
// Many rows: one workgroup to a CU (two splits for each CU's workgroup of 2048
// of 18432 cost 60 us in writing and joining them), down to splits of one tile:
// 4 chunks of 160 over 963, 8 + 8 heads of 128, take 40 us unsplit, 27 in
// splits of 256 keys at least, 22 of 64.  Tiles are counted from all rows, not
// from the longest sequence's.
AttentionShape attention_shape(uint32_t num_seqs, uint32_t total_q, uint32_t q_heads, uint32_t kv_heads,
                               uint32_t head_dim, uint32_t max_q_len, uint32_t max_context,
                               uint32_t window)
{
    AttentionShape r = {};
    const uint32_t group = q_heads / kv_heads;
    const uint64_t rows = (uint64_t)max_q_len * group;
    r.single = rows <= (uint64_t)kSingleRows;
    const uint32_t tile_rows = head_dim <= 128 ? TileShape<128>::kRows : TileShape<256>::kRows;
    r.tiles = r.single ? 1 : (uint32_t)((rows + tile_rows - 1) / tile_rows);
    // the keys that a workgroup's rows see
    const uint64_t span = r.single ? max_q_len : tile_rows / group + 2;
    uint64_t range = max_context;
    if (window > 0 && window + span < range)
        range = window + span;
    uint64_t blocks = (uint64_t)num_seqs * r.tiles;
    const uint64_t by_rows = (uint64_t)total_q * group / tile_rows + num_seqs;
    blocks = (r.single || blocks < by_rows ? blocks : by_rows) * kv_heads;
    blocks = blocks ? blocks : 1;
    uint64_t splits, unit;
    if (r.single) {
        unit = 128;
        splits = 2048 / blocks < range / 512 ? 2048 / blocks : range / 512;
        const uint64_t quick = 256 / blocks < range / unit ? 256 / blocks : range / unit;
        splits = splits > quick ? splits : quick;
    } else {
        unit = 64;   // a tile
        splits = 256 / blocks < range / unit ? 256 / blocks : range / unit;
    }
    splits = splits < kMaxSplits ? splits : kMaxSplits;
    splits = splits ? splits : 1;
    uint64_t keys = (range + splits - 1) / splits;
    keys = (keys + unit - 1) / unit * unit;
    keys = keys ? keys : unit;
    r.split_keys = (uint32_t)keys;
    r.splits = (uint32_t)((range + keys - 1) / keys);
    r.splits = r.splits ? r.splits : 1;
    if (r.splits > 1)
        r.workspace_bytes = (uint64_t)r.splits * total_q * q_heads * (head_dim + 2) * 4;
    return r;
}

hipError_t launch_attention(const AttentionArgs &a, const AttentionShape &shape, uint32_t num_seqs,
                            uint32_t dtype, uint32_t format, hipStream_t stream)
{
    if (dtype == KVCACHE_BF16)
        return attention_type<Bf16>(a, shape, num_seqs, format, stream);
    return attention_type<Fp16>(a, shape, num_seqs, format, stream);
}

}  // namespace kvc
