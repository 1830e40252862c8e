// Attention of new tokens (one, a chain or a tree of drafted ones) over the
// paged block-quantized cache (tq_tree_attention).
//
//   o[t] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t] . k_j),
//
// over the keys j that token t sees: all cached keys before the new tokens,
// and the new tokens its mask row names.  One pass over the keys with a
// running reference m in the exponent: p_j = 2^(c s_j - m), m raised (and the
// sums rescaled) only when some score passes it by 2^RAISE.
//
// Bound: a single token's step reads every cached byte once and is bound by
// HBM; trees multiply each dequantized key with many rows: the vector pipe
// (dequantization, softmax), LDS and the matrix cores are busy 45, 37 and 29 %
// of the trees' launch.  Measured (32 query heads, 8 key heads of 128, Q8_0 unless
// said): 64 sequences of 1600 to 16384 keys, one token: 229 us, 6.1 TB/s of
// cache (loads alone, nothing computed: 5.9; a plain read of the bytes: 7.1);
// one sequence of 8192 keys: 14 us, latency; 13 drafted tokens over 131000
// keys: 91 us in fp16 (k_attn_rows 92 and 5 joining when traced), 72 in bf16 (66,
// of which 15 start and store, and 5); 4 Q4_0 trees of up to 63 nodes over 20011
// keys: 62 us (58 and 11; each further key at 1.0 PFLOP/s, counting the rows of
// whole tiles).  A prompt's rows multiply all keys up to its end, twice what they
// see: 8192 tokens with none cached 1633 us, 337 TFLOP/s of what is seen.
//
// Split: rows are (token, query head) pairs of one key head, 16 per matrix
// tile, so a cached byte serves all the query heads and tokens of its head.
// Key steps of all sequences and heads are laid out in one line and cut into
// equal spans, one for each resident workgroup, so that unlike lengths cost
// little; where a cut falls inside a head's keys, k_attn_combine joins the
// sums.  Up to 32 rows (k_attn) the four waves of a workgroup
// hold the same rows and take every fourth group of 32 keys: keys and values
// go from memory through registers into the matrix cores
// (v_mfma_f32_16x16x32_f16), without LDS.  S^T = K Q^T leaves query columns in
// lanes and keys in registers, which is the operand layout of O^T = V^T P^T
// once lane group g's tokens are 4g..4g+3 of each 16 (cache_layout.h places
// the codes to match).  With more rows (k_attn_rows) the waves share the
// dequantized operands of 64 or 128 keys through LDS, stored as the fragments that
// the matrix instructions read.  Four row tiles a wave instead of two read
// LDS half as often but leave one wave per SIMD: 112 us for the 13 tokens in
// bf16, 106 for the trees (70 and 63 with two, both then), so two it is.
//
// Rounding: the queries enter as fp16 after a scaling of each row by a power
// of two that puts its largest element in [2^14, 2^15) (bf16 elements down to
// 2^-17 of that stay exact, below it they err by at most 2^-40 of the
// largest); code * scale of a key or value rounds once to fp16 (2^-11), as do
// the probabilities (taken times 2^BIAS against underflow: exact to 2^-11
// down to 2^-24 of the reference).  Scores, sums and outputs are fp32.  Beside
// a bf16 output's 2^-8 that is little (one token over 67 of 2047 pages of 64
// keys: errors of 0.0020 in root mean square, 0.0017 with nothing rounded but
// the output); with fp16 (FINE) only the values round so: a probability is two
// operands, itself and the rest of its rounding, and keys are exact (k_attn: a
// second operand with the rest, k_attn_rows: the codes as operands, the scales
// times the products in fp32).  The error is then 1.4
// times that of rounding exact outputs to fp16, 3.6 times without, where some
// channels of the keys are loud.  13 tokens over 131000 keys take 91 us so, 72
// without; k_attn, bound by HBM, takes no longer.  k_attn_rows with heads of 128
// then spills 3 to 22 of a lane's 256 registers, 16 to 60 bytes of scratch.
#include <algorithm>

#include "cache_layout.h"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int STEP = 32;                         // keys per wave and step
constexpr int STRIDE = STEP * WAVES;
constexpr float RAISE = 4.0f, BIAS = 10.0f;      // p <= 2^(RAISE + BIAS) = 2^14
constexpr float NO_REF = -3e38f;                 // near the lowest number: no score seen yet
// 2^22: half a step of fp32 is 1/4 there.  The branch for what lies past it costs
// those trees 1 us of 63, the 13 tokens under 1 and single tokens nothing; in one
// branch with the raise it needs more registers than there are (69 and 103 us).
constexpr float FAR = 4194304.0f;
constexpr int RED = 8;                           // fragments joined at a time
// What entering a head and row block costs, in keys, and the shortest span: one
// below that costs more to join than it saves (one token over 8192 keys: 15.6 us
// with 256, 14.8 with 512, 18.2 with 1024).  4 sequences of 20000 Q4_0 keys, 32
// tokens: 77.6 us when entering was not counted, 70.2 so.
constexpr int MIN_KEYS = 512;
// Up to this many heads and row blocks, one for each compute unit, k_attn_rows
// has one workgroup of eight waves there instead of two of four, and half as
// many parts are joined: those 4 sequences then take 66.6 us, and 32 of 2000
// Q8_0 keys and 16 tokens 42.0 instead of 50.0; but 64 of them 82.1 instead of
// 70.2, because starts and ends have nothing to run beside.
constexpr int FEW_UNITS = 256;
// From OWN_UNITS on the chip is filled four times over by a workgroup for each,
// and nothing is to be joined.
constexpr int OWN_UNITS = 2048;
// Of selected pages heads have about as many each: once they fill the chip
// (two workgroups a unit) each takes a workgroup, too.  Cut over workgroups / one each,
// 27 pages of 64, one token, us: 256 heads 28.7 / 23.2, 384 37.7 / 35.1, 504 43.0 / 40.4,
// 512 43.5 / 40.9, 520 49.2 / 51.8, 640 57.1 / 53.7, 768 66.8 / 59.4, 1024 80.7 / 76.9, 1520
// 119.8 / 111.0.  Where all but one sequence in eight are too short for pages to be
// left out that is the other way round: 384 heads 24.8 / 29.2, 768 38.1 / 41.4, 1520 65.8 /
// 69.0; with 67 pages 384 heads 36.7 / 59.5, 512 47.8 / 63.2, 1024 78.4 / 102.4.
constexpr int EVEN_UNITS = 512;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

template <int CT, int D> struct Geo {
    static constexpr int NB = D / 32;            // 32-element blocks = matrix steps of Q K^T
    static constexpr int NT = D / 16;            // 16-element tiles of the output
    static constexpr int KW = CT == TQ_Q8_0 ? D / 16 : D / 32;   // code dwords per lane and 16 keys
    // values: elements next to each other in a lane, and 16 * CW apart
    static constexpr int CW = CT == TQ_Q8_0 ? (D % 64 == 0 ? 4 : 2)
                                            : (D % 128 == 0 ? 8 : (D % 64 == 0 ? 4 : 2));
    static constexpr int NH = D / (16 * CW);
    static constexpr int VL = CT == TQ_Q8_0 ? CW : CW / 2;       // code dwords per load
    static constexpr int TB = (int)token_code_bytes(CT, D);
};

// 16 keys' codes and scales as one lane loads them.
template <int CT, int D> struct Tile {
    using G = Geo<CT, D>;
    uint32_t k[G::KW], ks[(G::NB + 1) / 2];
    uint32_t v[G::KW];
    uint32_t vs[2 * G::NH];
};

// N dwords (aligned to 4 N bytes, N = 3 to 4) at byte v + s of a buffer, v per
// lane and s uniform; zeros past its end.  AUX: BUF_NT where no other
// workgroup reads the same keys (one row block): 64 sequences of one token
// 262 -> 241 us; with two row blocks the caches serve the second.
template <int N, int AUX>
__device__ __forceinline__ void load_words(uint32_t *w, __amdgpu_buffer_rsrc_t b, int v, int s)
{
    if constexpr (N == 4) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b128(b, v, s, AUX);
        w[0] = x[0]; w[1] = x[1]; w[2] = x[2]; w[3] = x[3];
    } else if constexpr (N == 3) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b96(b, v, s, AUX);
        w[0] = x[0]; w[1] = x[1]; w[2] = x[2];
    } else if constexpr (N == 2) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b64(b, v, s, AUX);
        w[0] = x[0]; w[1] = x[1];
    } else {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, v, s, AUX);
    }
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A read-only word at a uniform address, through the scalar cache: it does
// not wait behind the tile loads in flight.
__device__ __forceinline__ int load_uniform(const int32_t *p)
{
    return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}

// Where the keys of one sequence and key head lie (all uniform).
struct Place {
    const int32_t *table;
    uint64_t k, v;                   // of page 0's chunk
    uint32_t stride, pages;          // bytes from page to page
    int bytes, log_page, last, end;  // of a chunk; the table's last entry; keys end before `end`
    int plain;                       // keys before it are cached ones of the range
};

// The page table's entry for a key.  No branch: a load that may not happen
// would make every wait for the tile loads in flight wait for all of them.
__device__ __forceinline__ int entry_at(const Place &c, int key)
{
    return load_uniform(c.table + min(key >> c.log_page, c.last));
}

__device__ __forceinline__ bool mapped(const Place &c, int entry, int key)
{
    return key < c.end && (uint32_t)entry < c.pages;
}

// The chunks of one page; of no bytes where there is none or the keys have
// ended, so that its loads read zeros and move nothing.
struct Chunks {
    __amdgpu_buffer_rsrc_t k, v;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(uint64_t at, int n)
{
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)at), hi = (uint32_t)uniform((int)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(((uint64_t)hi << 32) | lo), (short)0,
                                             uniform(n), 0x00020000);
}

__device__ __forceinline__ Chunks chunks_at(const Place &c, int entry, int key)
{
    const bool there = mapped(c, entry, key);
    const int n = there ? c.bytes : 0;
    const uint64_t at = (uint64_t)(there ? (uint32_t)entry : 0) * c.stride;
    return Chunks{chunk_rsrc(c.k + at, n), chunk_rsrc(c.v + at, n)};
}

// The 16 keys at position pos (uniform) of a page, and their values.
template <int CT, int D, int AUX>
__device__ __forceinline__ void load_keys(Tile<CT, D> &raw, const Chunks &c, int pos, int P,
                                          int lane)
{
    using G = Geo<CT, D>;
    const int r = lane & 15;
    constexpr int B = k_piece<CT, D>();
#pragma unroll
    for (int n = 0; n < G::KW * 4 / B; n++)
        load_words<B / 4, AUX>(raw.k + n * (B / 4), c.k, lane * B + n * (64 * B), pos * G::TB);
    const int scales = P * G::TB;
    if constexpr (G::NB == 3) {
        raw.ks[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(c.k, r * 6, scales + pos * 6, AUX) |
                    (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(c.k, r * 6 + 2,
                                                                             scales + pos * 6, AUX) << 16;
        raw.ks[1] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(c.k, r * 6 + 4, scales + pos * 6, AUX);
    } else {
        load_words<G::NB / 2, AUX>(raw.ks, c.k, r * (G::NB * 2), scales + pos * (G::NB * 2));
    }
}

template <int CT, int D, int AUX>
__device__ __forceinline__ void load_values(Tile<CT, D> &raw, const Chunks &c, int pos, int P,
                                            int lane)
{
    using G = Geo<CT, D>;
    const int r = lane & 15, g = lane >> 4, scales = P * G::TB;
    const int vl = g * (4 * G::TB) + r * (G::VL * 4);
    const int sl = ((G::CW * r / 32) * P + 4 * g) * 2;
#pragma unroll
    for (int h = 0; h < G::NH; h++) {
        load_words<G::VL, AUX>(raw.v + h * G::VL, c.v, vl + h * (64 * G::VL), pos * G::TB);
        // 16 * CW elements further: CW / 2 blocks of P scales
        load_words<2, AUX>(raw.vs + 2 * h, c.v, sl, scales + pos * 2 + h * G::CW * P);
    }
}

template <int CT, int D, int AUX>
__device__ __forceinline__ void load_tile(Tile<CT, D> &raw, const Chunks &c, int pos, int P,
                                          int lane)
{
    load_keys<CT, D, AUX>(raw, c, pos, P, lane);
    load_values<CT, D, AUX>(raw, c, pos, P, lane);
}

__device__ __forceinline__ h2 as_h2(uint32_t w) { return __builtin_bit_cast(h2, w); }
__device__ __forceinline__ uint32_t as_u32(h2 h) { return __builtin_bit_cast(uint32_t, h); }

// Codes to fp16 pairs: with 0x64 above it a byte u reads 1024 + u, so one
// subtraction gives the signed code exactly.
__device__ __forceinline__ void codes8(uint32_t w, h2 &a, h2 &b)
{
    const h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    a = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
    b = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
}

__device__ __forceinline__ h2 codes4(uint32_t w)
{
    const h2 off = {(_Float16)1032.0f, (_Float16)1032.0f};
    // one three-input operation: the mask in a vector register, the bits in a
    // scalar one (two literals would be two operations)
    uint32_t mask = 0x000f000fu, bits = 0x64006400u;
    asm("" : "+v"(mask));
    asm("" : "+s"(bits));
    return as_h2((w & mask) | bits) - off;
}

union Frag {
    h2 p[4];
    h8 v;
};

// Block s of the lane's key: the codes of 8 elements, and the scale.
template <int CT, int D>
__device__ __forceinline__ Frag key_codes(const Tile<CT, D> &raw, int s)
{
    Frag f;
    if constexpr (CT == TQ_Q8_0) {
        codes8(raw.k[2 * s], f.p[0], f.p[1]);
        codes8(raw.k[2 * s + 1], f.p[2], f.p[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            f.p[i] = codes4(raw.k[s] >> (4 * i));
    }
    return f;
}

template <int CT, int D>
__device__ __forceinline__ h2 key_scale(const Tile<CT, D> &raw, int s)
{
    const h2 two = as_h2(raw.ks[s >> 1]);
    return s & 1 ? two.yy : two.xx;
}

template <int CT, int D>
__device__ __forceinline__ h8 key_frag(const Tile<CT, D> &raw, int s)
{
    Frag f = key_codes<CT, D>(raw, s);
    const h2 dd = key_scale<CT, D>(raw, s);
#pragma unroll
    for (int i = 0; i < 4; i++)
        f.p[i] *= dd;
    return f.v;
}

// Output tile t's element of the lane: 4 tokens.
template <int CT, int D>
__device__ __forceinline__ void value_half(const Tile<CT, D> &raw, int t, h2 &a, h2 &b)
{
    using G = Geo<CT, D>;
    const int h = t / G::CW, j = t % G::CW;
    if constexpr (CT == TQ_Q8_0) {
        codes8(raw.v[h * G::VL + j], a, b);
    } else {
        const uint32_t w = raw.v[h * G::VL + (j >> 1)] >> (4 * (j & 1));
        a = codes4(w);
        b = codes4(w >> 8);
    }
    a *= as_h2(raw.vs[2 * h]);
    b *= as_h2(raw.vs[2 * h + 1]);
}

// What the value blocks of a tile hold must not meet a probability of 0 as
// NaN or infinity: of the lane's four tokens (keys key .. key + 3), those not
// there count as zeros, and so do new ones whose scale is no number.
template <int CT, int D>
__device__ __forceinline__ void drop_values(Tile<CT, D> &raw, int key, bool there, int ctx, int L)
{
    const int left = there ? L - key : 0;        // tokens of the four that are there
    auto keep = [&](uint32_t w, int k) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t e = 0x7C00u << (16 * i);
            const int odd = (int)(key + k + i >= ctx) & (int)((w & e) == e);
            m |= (int)(k + i < left) & (odd ^ 1) ? 0xFFFFu << (16 * i) : 0u;
        }
        return w & m;
    };
#pragma unroll
    for (int h = 0; h < 2 * Geo<CT, D>::NH; h++)
        raw.vs[h] = keep(raw.vs[h], 2 * (h & 1));
}

// x, which the compiler takes for a new value: what is derived from it is not
// kept in registers from one turn of an outer loop to the next.
__device__ __forceinline__ int fresh(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// Sums of cut rows: outputs (fragments of a slot), reference and sum of each
// row, and for each sequence, key head and row block its first slot and how
// many parts it has.
struct Parts {
    f4 *sum;
    float2 *ml;
    int2 *list;
};

struct Launch {
    AttnArgs a;
    AttnPlan p;
    Parts parts;
};

// The kernel's argument, read anew: what one phase of a kernel has loaded of
// it is not kept in scalar registers through the others.
__device__ __forceinline__ const Launch &arguments()
{
    auto p = __builtin_amdgcn_kernarg_segment_ptr();     // in the constant address space
    asm volatile("" : "+s"(p));
    return *(const Launch *)p;
}

// One sequence, and key head h and row block rb of it; row r is (token
// r / group, query head h * group + r % group).
struct Rows {
    int b, h, rb, T, ctx, L;
    int64_t tok0;
};

// Lengths and starts are held inside the buffers whatever they say.
__device__ __forceinline__ void set_lengths(Rows &w, const AttnArgs &a, int s0, int s1, int ctx)
{
    const int64_t t0 = min(max((int64_t)s0, (int64_t)0), a.tokens);
    const int64_t t1 = min((int64_t)s1, a.tokens);
    w.tok0 = t0;
    w.T = (int)min(max(t1 - t0, (int64_t)0), (int64_t)a.max_nodes);
    w.ctx = max(ctx, 0);
    const int64_t most = (int64_t)a.table_pages << a.log_page;
    w.L = (int)min((int64_t)w.ctx + w.T, most);
}

__device__ __forceinline__ Rows rows_of(const AttnArgs &a, int b)
{
    Rows w;
    w.b = b;
    w.h = w.rb = 0;
    set_lengths(w, a, load_uniform(a.starts + b), load_uniform(a.starts + b + 1),
                load_uniform(a.ctx + b));
    return w;
}

// Key steps of `keys` keys, and row blocks, of a sequence.  One that has new
// tokens takes a step even if it sees no key: its outputs are zeros.
__device__ __forceinline__ int steps_of(const Rows &w, int keys)
{
    return w.T == 0 ? 0 : max((w.L + keys - 1) / keys, 1);
}

__device__ __forceinline__ int blocks_of(const AttnArgs &a, const AttnPlan &p, const Rows &w)
{
    return (w.T * a.group + p.tiles * 16 - 1) / (p.tiles * 16);
}

// The line of key steps runs sequence by sequence, in it (head, row block) by
// (head, row block): a lane's sequence (none past the batch), its (head, row
// block)s and the steps of one.
struct Entry {
    int s0, s1, ctx, steps, units;
};

__device__ __forceinline__ Entry line_entry(const AttnArgs &a, const AttnPlan &p, int keys, int b)
{
    Entry e{0, 0, 0, 0, 0};
    if (b < a.batch) {
        e.s0 = a.starts[b];
        e.s1 = a.starts[b + 1];
        e.ctx = a.ctx[b];
    }
    Rows w;
    set_lengths(w, a, e.s0, e.s1, e.ctx);
    if (b < a.batch) {
        e.steps = steps_of(w, keys);
        e.units = blocks_of(a, p, w) * a.kv_heads;
    }
    return e;
}

template <int CTRL, int ROWS> __device__ __forceinline__ int64_t dpp64(int64_t x)
{
    const int lo = __builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), CTRL, ROWS, 0xF, true);
    return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// Running sum over the lanes: shifts by 1, 2, 4, 8 in each row of 16, then
// the last lane of a row added to the rows behind it.
__device__ __forceinline__ int64_t scan_lanes(int64_t v)
{
    v += dpp64<0x111, 0xF>(v);
    v += dpp64<0x112, 0xF>(v);
    v += dpp64<0x114, 0xF>(v);
    v += dpp64<0x118, 0xF>(v);
    v += dpp64<0x142, 0xA>(v);
    v += dpp64<0x143, 0xC>(v);
    return v;
}

__device__ __forceinline__ int lane_of(int x, int k) { return __builtin_amdgcn_readlane(x, k); }

__device__ __forceinline__ int64_t lane_of(int64_t x, int k)
{
    return (int64_t)(((uint64_t)(uint32_t)lane_of((int)(x >> 32), k) << 32) |
                     (uint32_t)lane_of((int)x, k));
}

// Steps for each workgroup of a line of `all` (it has less than 2048 * 2^24
// steps, and 512 workgroups share a long one).
__device__ __forceinline__ int span_for(int64_t all, const AttnPlan &p)
{
    const uint32_t groups = p.groups;
    return (int)max(all < (int64_t(1) << 31) ? (uint32_t)((uint32_t)all + groups - 1) / groups
                                             : (uint32_t)((all + groups - 1) / groups),
                    1u);
}

// A workgroup's place in the line: its next steps are `step` .. of (head, row
// block) `q` of the sequence in w, `left` steps remain, of which going on to
// the next (head, row block) takes `enter`.
struct Cursor {
    Rows w;
    int q, steps, blocks, step, left, span, enter;
};

__device__ __forceinline__ void set_sequence(Cursor &c, const AttnArgs &a, const AttnPlan &p,
                                             int keys, const Rows &w)
{
    c.w = w;
    c.steps = steps_of(w, keys);
    c.blocks = blocks_of(a, p, w);
}

// Key head h and row block rb of sequence b (none where b is the batch).
struct Unit {
    int b, h, rb;
};

// Every sequence has the row blocks of max_nodes tokens.
__device__ __forceinline__ Unit unit_of(const AttnArgs &a, const AttnPlan &p, uint32_t unit)
{
    const uint32_t per = (uint32_t)a.kv_heads * p.row_blocks, b = unit / per, q = unit - b * per;
    const uint32_t h = q / p.row_blocks;
    return {(int)min(b, (uint32_t)a.batch), (int)h, (int)(q - h * p.row_blocks)};
}

// Row blocks in the order of the rows, where max_nodes is far above what
// sequences have.  With x(b) = rows before sequence b / rows of a block, its
// row blocks, ceil(x(b + 1) - x(b)) at most, fit between first(b) = floor(x(b))
// + b and first(b + 1), whatever the lengths: no sum over sequences is needed,
// and a wave finds b in three turns of 64 looks.  Starts that go back lead to
// some sequence inside the batch.
__device__ __forceinline__ Unit unit_by_rows(const AttnArgs &a, const AttnPlan &p, uint32_t unit,
                                             int lane)
{
    const uint32_t v = unit / (uint32_t)a.kv_heads;
    auto first = [&](int b) {
        const uint32_t t = (uint32_t)min(max((int64_t)a.starts[b], (int64_t)0), a.tokens);
        return t * (uint32_t)a.group / (uint32_t)(p.tiles * 16) + (uint32_t)b;
    };
    int lo = 0, hi = a.batch;                    // lo <= b < hi
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6, b = lo + lane * step;
        const uint64_t after = __ballot(b >= hi || first(b) > v);
        const int k = after ? __builtin_ctzll(after) : 64;
        if (k == 0)
            return {a.batch, 0, 0};              // rows before the first sequence
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
    }
    const uint32_t f0 = (uint32_t)uniform((int)first(lo)), f1 = (uint32_t)uniform((int)first(lo + 1));
    if (v < f0 || v >= f1)
        return {a.batch, 0, 0};
    const uint32_t n = f1 - f0, q = unit - f0 * (uint32_t)a.kv_heads, h = q / n;
    return {lo, (int)h, (int)(q - h * n)};
}

__device__ __forceinline__ Cursor first_span(const AttnArgs &a, const AttnPlan &p, int keys,
                                             int lane)
{
    Cursor c;
    c.left = c.enter = 0;
    if (p.groups == 0) {
        // many heads: one workgroup for all the keys of each
        const uint32_t unit = blockIdx.y * gridDim.x + blockIdx.x;
        const Unit u = p.by_rows ? unit_by_rows(a, p, unit, lane) : unit_of(a, p, unit);
        if (u.b >= a.batch)
            return c;
        set_sequence(c, a, p, keys, rows_of(a, u.b));
        c.q = u.h * c.blocks + u.rb;
        c.step = 0;
        if (u.h < a.kv_heads && u.rb < c.blocks)
            c.left = c.steps;
        return c;
    }
    // To enter a (head, row block), with its lengths, rows, sums and outputs,
    // takes about as long as MIN_KEYS of its keys, so the line has that many
    // in front of each.  Where all have as many steps, each may be cut by
    // itself for the workgroups there are for it, if no span gets longer:
    // then none enters two.
    c.enter = MIN_KEYS / keys;
    auto cut_alike = [&](int steps, int64_t units) {
        if (units > p.groups)
            return false;
        const uint32_t n = (uint32_t)p.groups / (uint32_t)units, cut = (steps + n - 1) / n;
        if ((int64_t)(cut - 1) * p.groups >= (steps + c.enter) * units)
            return false;
        c.q = (int)(blockIdx.x / n);
        c.step = (int)((blockIdx.x - c.q * n) * cut);
        c.enter = 0;
        c.span = (int)cut;
        c.left = c.q < units ? min(c.span, steps - c.step) : 0;
        return true;
    };
    int64_t at;
    if (a.batch == 1) {
        set_sequence(c, a, p, keys, rows_of(a, 0));
        const int64_t units = (int64_t)c.blocks * a.kv_heads, all = (c.steps + c.enter) * units;
        if (units == 0 || cut_alike(c.steps, units))
            return c;
        c.span = span_for(all, p);
        at = (int64_t)blockIdx.x * c.span;
        if (at >= all)
            return c;
    } else {
        // by 64 sequences in the lanes; the first 64 are read once
        auto steps_in = [&](const Entry &e) { return (int64_t)(e.steps + c.enter) * e.units; };
        auto sequence = [&](const Entry &e, int base, int k) {
            Rows w;
            w.b = base + k;
            w.h = w.rb = 0;
            set_lengths(w, a, lane_of(e.s0, k), lane_of(e.s1, k), lane_of(e.ctx, k));
            set_sequence(c, a, p, keys, w);
        };
        Entry e = line_entry(a, p, keys, lane);
        const int steps0 = lane_of(e.steps, 0), units0 = lane_of(e.units, 0);
        if (units0 && a.batch <= 64 &&
            !__any(lane < a.batch && (e.steps != steps0 || e.units != units0)) &&
            cut_alike(steps0, (int64_t)units0 * a.batch)) {
            if (c.left > 0) {
                const int k = (int)((uint32_t)c.q / (uint32_t)units0);
                c.q -= k * units0;
                sequence(e, 0, k);
            }
            return c;
        }
        int64_t end = scan_lanes(steps_in(e)), all = lane_of(end, 63);
        for (int base = 64; base < a.batch; base += 64)
            all += lane_of(scan_lanes(steps_in(line_entry(a, p, keys, base + lane))), 63);
        c.span = span_for(all, p);
        at = (int64_t)blockIdx.x * c.span;
        if (at >= all)
            return c;
        int base = 0;
        uint64_t hit = __ballot(at < end);
        while (!hit) {                           // found before the batch ends: at < all
            at -= lane_of(end, 63);
            base += 64;
            e = line_entry(a, p, keys, base + lane);
            end = scan_lanes(steps_in(e));
            hit = __ballot(at < end);
        }
        const int k = __builtin_ctzll(hit);
        at -= lane_of(end - steps_in(e), k);
        sequence(e, base, k);
    }
    // positions inside a sequence pass 31 bits only past 2^31 steps of it
    const int each = c.steps + c.enter;
    c.q = at < (int64_t(1) << 31) ? (int)((uint32_t)at / (uint32_t)each) : (int)(at / each);
    const int place = (int)(at - (int64_t)c.q * each) - c.enter;
    c.step = max(place, 0);
    c.left = c.span + min(place, 0);
    return c;
}

// What a workgroup does next: keys begin .. end - 1 of the rows in w, the
// first of `parts` parts if begin is 0; `whole` if those are all the rows
// have, else its sums go to slot `slot`: two a workgroup, the even one for its
// first rows (part n > 0 of any rows), the odd one for its last.
struct Work {
    Rows w;
    bool whole;
    int slot, parts, begin, end;
};

// false: nothing is left.
__device__ __forceinline__ bool next_work(Cursor &c, Work &k, const Launch &launch, int keys,
                                          bool first)
{
    const AttnArgs &a = launch.a;
    const AttnPlan &p = launch.p;
    if (!first) {
        if (c.left <= 0 || p.groups == 0)
            return false;
        c.step = 0;
        c.left -= c.enter;
        if (++c.q == c.blocks * a.kv_heads) {
            c.q = 0;
            int b = c.w.b;
            do {
                if (++b >= a.batch)
                    return false;
                set_sequence(c, a, p, keys, rows_of(a, b));
            } while (c.steps == 0);
        }
    }
    if (c.left <= 0)
        return false;
    const int take = min(c.left, c.steps - c.step);
    k.w = c.w;
    k.w.h = c.q / c.blocks;
    k.w.rb = c.q - k.w.h * c.blocks;
    k.whole = take == c.steps;
    k.parts = k.whole ? 1 : 1 + (c.steps - take + c.span - 1) / c.span;
    k.slot = 2 * blockIdx.x + !first;
    k.begin = c.step * keys;
    k.end = min(c.w.L, (c.step + take) * keys);
    c.left -= take;
    return true;
}

// Fragment (16-row tile, output tile t) of a row block, as every wave holds
// it: lane's row lane & 15, elements of rows 4 (lane >> 4) + 0..3 of the tile.
template <int CT, int D>
__device__ __forceinline__ void store_frag(const AttnArgs &a, const Rows &w, int tiles, int tile,
                                           int t, int lane, f4 o)
{
    using G = Geo<CT, D>;
    const int r = (w.rb * tiles + tile) * 16 + (lane & 15);
    if (r >= w.T * a.group)
        return;
    const int node = r / a.group;
    const int64_t at = (w.tok0 + node) * a.yts + (w.h * a.group + r - node * a.group) * a.yhs;
    const int d0 = 16 * G::CW * (t / G::CW) + t % G::CW + 4 * (lane >> 4) * G::CW;
    uint16_t *y = (uint16_t *)a.y + at + d0;
#pragma unroll
    for (int e = 0; e < 4; e++)
        y[G::CW * e] = a.dtype == TQ_BF16 ? f32_to_16<TQ_BF16>(o[e]) : f32_to_16<TQ_F16>(o[e]);
}

// One 16-row tile of a wave: queries in fp16 after the row's power of two, c
// = what a score is times, and the running sums.
template <int D> struct Query {
    h8 q[D / 32];
    float c, m;
    int node, far;                               // far: some row's reference is (uniform)
    f4 l, o[D / 16];                             // l: the sum in each element
};

template <int D>
__device__ __forceinline__ void load_query(Query<D> &x, const AttnArgs &a, const Rows &w, int tiles,
                                           int tile, int lane)
{
    constexpr int NB = D / 32;
    const int g = lane >> 4, r = (w.rb * tiles + tile) * 16 + (lane & 15);
    const bool live = r < w.T * a.group;
    x.node = live ? r / a.group : 0;
    const int64_t at =
        (w.tok0 + x.node) * a.qts + (w.h * a.group + (live ? r - x.node * a.group : 0)) * a.qhs;
    float v[NB][8], big = 0.0f;
#pragma unroll
    for (int s = 0; s < NB; s++) {
        if (a.dtype == TQ_BF16)
            load_x8<TQ_BF16>(v[s], a.q, at + 32 * s + 8 * g);
        else
            load_x8<TQ_F16>(v[s], a.q, at + 32 * s + 8 * g);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[s][e] = live ? v[s][e] : 0.0f;
            big = fmaxf(big, fabsf(v[s][e]));
        }
    }
    big = fmaxf(big, __shfl_xor(big, 16));
    big = fmaxf(big, __shfl_xor(big, 32));
    // 2^k with big * 2^k in [2^14, 2^15); 1 for a row of zeros or with an infinity
    const int ex = (int)(__builtin_bit_cast(uint32_t, big) >> 23);
    const int k = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -126), 126);
    const float up = __builtin_bit_cast(float, (uint32_t)(127 + k) << 23);
    const float down = __builtin_bit_cast(float, (uint32_t)(127 - k) << 23);
#pragma unroll
    for (int s = 0; s < NB; s++)
#pragma unroll
        for (int e = 0; e < 8; e++)
            x.q[s][e] = (_Float16)(v[s][e] * up);
    // not 0, which would make a number of the -inf of a key that is not seen
    x.c = fmaxf(a.scale * 1.44269504088896f * down, 0x1p-126f);
    x.m = NO_REF;
    x.far = 0;
    x.l = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < D / 16; t++)
        x.o[t] = f4{0.0f, 0.0f, 0.0f, 0.0f};
}

// Which of the keys key .. key + 3 token `node` sees, as 4 bits: all cached
// ones, new ones by its mask row (or up to itself), none past the end or on a
// page that is not there.
__device__ __forceinline__ uint32_t seen4(const AttnArgs &a, const Rows &w, int node, int key,
                                          bool there)
{
    const int n = max(key - w.ctx, -4);
    uint32_t bits;
    if (a.mask) {
        const uint32_t *row = a.mask + (w.tok0 + node) * a.mask_stride;
        const int first = max(n, 0) >> 5, last = first + 1;
        const uint32_t lo = row[min(first, a.mask_words - 1)];
        const uint32_t hi = row[min(last, a.mask_words - 1)];
        const uint64_t both = (first < a.mask_words ? (uint64_t)lo : 0) |
                              (last < a.mask_words ? (uint64_t)hi << 32 : 0);
        bits = (uint32_t)(both >> (max(n, 0) & 31));
    } else {
        bits = (1u << min(max(node - max(n, 0) + 1, 0), 4)) - 1;
    }
    const int before = max(-n, 0);               // keys of the four that are cached
    bits = (bits << before) | ((1u << before) - 1);
    const int left = min(max(w.L - key, 0), 4);
    return there ? bits & ((1u << left) - 1) : 0;
}

// Scores of 32 keys from kb (some are new tokens, past the end, or on pages
// that are not there): -inf where not seen.
template <int D>
__device__ __forceinline__ void mask_scores(f4 (&s)[2], const Query<D> &x, const AttnArgs &a,
                                            const Rows &w, int kb, bool oka, bool okb, int g)
{
    const uint32_t b0 = seen4(a, w, x.node, kb + 4 * g, oka);
    const uint32_t b1 = seen4(a, w, x.node, kb + 16 + 4 * g, okb);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        s[0][e] = (b0 >> e) & 1 ? s[0][e] : -__builtin_inff();
        s[1][e] = (b1 >> e) & 1 ? s[1][e] : -__builtin_inff();
    }
}

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The exponent where the reference is so large that fp32's steps there, which
// a product rounded only with the sum would be off the reference by, are no
// longer small: the product rounded by itself, as the reference was, so that
// none passes it by more than RAISE.
__device__ __forceinline__ float far_exponent(float s, float c, float m)
{
#pragma clang fp contract(off)
    const float x = s * c;
    return (x - m) + BIAS;
}

// Probabilities of 32 keys as the operand of the second product; the
// reference, sum and outputs follow where a score passes it.  The sum is one
// more product, with a row of ones: it then adds the rounded probabilities,
// the same ones that weigh the values.
template <int D, bool FINE>
__device__ __forceinline__ h8 softmax_step(const f4 (&s)[2], Query<D> &x, h8 &rest)
{
    // the median with +inf: a maximum without fmaxf's extra operation on each
    // product of the matrix cores (a NaN score shows in p, not here)
    float inf = __builtin_inff();
    asm("" : "+s"(inf));
    auto larger = [&](float a, float b) { return __builtin_amdgcn_fmed3f(a, b, inf); };
    float top = larger(larger(larger(s[0][0], s[0][1]), larger(s[0][2], s[0][3])),
                       larger(larger(s[1][0], s[1][1]), larger(s[1][2], s[1][3])));
    top *= x.c;
    if (__any(top > x.m + RAISE)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(x.m, top);
        const float f = __builtin_amdgcn_exp2f(x.m - mn);
        x.m = mn;
        // (an infinite one has no way out, and its neighbours stay as they are)
        x.far = uniform(__any(fabsf(mn) > FAR && fabsf(mn) < __builtin_inff() && mn != NO_REF));
        x.l *= f;
#pragma unroll
        for (int t = 0; t < D / 16; t++)
            x.o[t] *= f;
    }
    const float ref = BIAS - x.m;
    float z[2][4];
    if (__builtin_expect(x.far, 0)) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            z[i >> 2][i & 3] = far_exponent(s[i >> 2][i & 3], x.c, x.m);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            z[i >> 2][i & 3] = fmaf(s[i >> 2][i & 3], x.c, ref);
    }
    Frag p, r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int T = i >> 1, e = 2 * (i & 1);
        const f2 y = {__builtin_amdgcn_exp2f(z[T][e]), __builtin_amdgcn_exp2f(z[T][e + 1])};
        p.p[i] = __builtin_convertvector(y, h2);
        if constexpr (FINE)
            r.p[i] = __builtin_convertvector(
                (f2{y[0] - (float)p.p[i][0], y[1] - (float)p.p[i][1]}), h2);
    }
    const _Float16 one = (_Float16)1.0f;
    const h8 ones = {one, one, one, one, one, one, one, one};
    x.l = mfma(ones, p.v, x.l);
    if constexpr (FINE) {
        x.l = mfma(ones, r.v, x.l);
        rest = r.v;
    }
    return p.v;
}

// Joins the KG waves that hold the same rows (rg, of RG groups) and stores
// the outputs, or their sums where other workgroups have more of the keys.  red: RED
// fragments of 64 lanes per wave.
template <int CT, int D, int QT, int RG, int KG>
__device__ __forceinline__ void finish(Query<D> (&x)[QT], const Launch &launch, const Work &k,
                                       int rg, int kg, int lane, f4 *red, float *ml)
{
    const AttnArgs &a = launch.a;
    const AttnPlan &p = launch.p;
    const Parts &parts = launch.parts;
    lane = fresh(lane);
    constexpr int NT = D / 16, TILES = RG * QT, F = TILES * NT, MINE = QT * NT;
    const int col = lane & 15, g = lane >> 4;
    float f[QT], l[QT];
#pragma unroll
    for (int i = 0; i < QT; i++) {
        l[i] = x[i].l[0];
        f[i] = 1.0f;
    }
    __syncthreads();                             // the fragments' region is free
    if constexpr (KG > 1) {
        const int mine = ((rg * KG + kg) * QT * 16 + col) * 2;
        if (g == 0)
#pragma unroll
            for (int i = 0; i < QT; i++) {
                ml[mine + i * 32] = x[i].m;
                ml[mine + i * 32 + 1] = l[i];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < QT; i++) {
            const float *q = ml + (rg * KG * QT * 16 + i * 16 + col) * 2;
            float mm = NO_REF, ll = 0.0f;
#pragma unroll
            for (int n = 0; n < KG; n++)
                mm = fmaxf(mm, q[n * QT * 32]);
#pragma unroll
            for (int n = 0; n < KG; n++)
                ll += q[n * QT * 32 + 1] * __builtin_amdgcn_exp2f(q[n * QT * 32] - mm);
            f[i] = __builtin_amdgcn_exp2f(x[i].m - mm);
            x[i].m = mm;
            l[i] = ll;
        }
    }
    const int64_t slot = k.slot;
    if (parts.list && k.begin == 0 && threadIdx.x == 0)
        parts.list[(k.w.b * a.kv_heads + k.w.h) * p.row_blocks + k.w.rb] = make_int2(k.slot, k.parts);
    if (!k.whole && kg == 0 && g == 0) {
#pragma unroll
        for (int i = 0; i < QT; i++) {
            float2 *q = parts.ml + slot * (TILES * 16) + (rg * QT + i) * 16 + col;
            *q = make_float2(x[i].m, l[i]);
        }
    }
    // The fragments pass through LDS, RED of a wave at a time, so that what
    // is done with each is a loop: this code runs once, and a cold line of
    // code costs more than the loop.
    f4 *own = red + (rg * KG + kg) * (RED * 64) + lane, *group = red + rg * KG * (RED * 64) + lane;
    constexpr int SHARE = RED / KG;
#pragma unroll
    for (int f0 = 0; f0 < MINE; f0 += RED) {
        if (KG > 1 && f0)
            __syncthreads();
#pragma unroll
        for (int n = 0; n < RED; n++)
            if (f0 + n < MINE)
                own[n * 64] = x[(f0 + n) / NT].o[(f0 + n) % NT] * f[(f0 + n) / NT];
        if (KG > 1)
            __syncthreads();
#pragma unroll 1
        for (int n = kg * SHARE; n < min((kg + 1) * SHARE, MINE - f0); n++) {
            f4 sum = group[n * 64];
#pragma unroll
            for (int e = 1; e < KG; e++)
                sum += group[(e * RED + n) * 64];
            const int i = (f0 + n) / NT, t = (f0 + n) % NT;
            if (!k.whole) {
                // rows past the tokens have no part
                if ((k.w.rb * TILES + rg * QT + i) * 16 + col < k.w.T * a.group)
                    parts.sum[(slot * F + (rg * QT + i) * NT + t) * 64 + lane] = sum;
            } else {
                float li = l[0];
#pragma unroll
                for (int e = 1; e < QT; e++)
                    li = i == e ? l[e] : li;
                // nothing seen: zeros
                store_frag<CT, D>(a, k.w, TILES, rg * QT + i, t, lane,
                                  li == 0.0f ? f4{0, 0, 0, 0} : sum * (1.0f / li));
            }
        }
    }
}

template <int CT, int D>
__device__ __forceinline__ Place place_of(const AttnArgs &a, const Work &k)
{
    Place c;
    c.table = a.table + k.w.b * a.table_stride + k.w.h * a.table_head_stride;
    c.bytes = (int)chunk_bytes(CT, D, 1 << a.log_page);
    c.stride = (uint32_t)a.kv_heads * c.bytes;
    c.k = (uint64_t)a.kc + (uint32_t)(k.w.h * c.bytes);
    c.v = (uint64_t)a.vc + (uint32_t)(k.w.h * c.bytes);
    c.pages = (uint32_t)a.pages;
    c.log_page = a.log_page;
    c.last = a.table_pages - 1;
    c.end = k.end;
    c.plain = min(k.w.ctx, k.end);
    return c;
}

// Whether all pages of keys begin .. end - 1 are there.
__device__ __forceinline__ bool all_mapped(const Place &c, int begin, int lane)
{
    bool bad = false;
    for (int i = (begin >> c.log_page) + lane; i <= (c.end - 1) >> c.log_page; i += 64)
        bad = bad || (uint32_t)c.table[i] >= c.pages;
    return !__any(bad);
}

// Up to 32 rows: every wave has its own keys.
template <int CT, int D, int QT, bool FINE>
__global__ __launch_bounds__(THREADS, D <= 128 || CT == TQ_Q4_0 ? 2 : 1) void k_attn(
    Launch launch)
{
    using G = Geo<CT, D>;
    __shared__ f4 red[WAVES * RED * 64];
    __shared__ float ml[WAVES * QT * 16 * 2];
    const int lane0 = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int P = 1 << launch.a.log_page;
    Cursor cur = first_span(launch.a, launch.p, STRIDE, lane0);
    Work k;
    for (bool first = true; next_work(cur, k, arguments(), STRIDE, first); first = false) {
        const Rows &w = k.w;
        const AttnArgs &a = arguments().a;
        const int lane = fresh(lane0), g = lane >> 4;
        const Place pl = place_of<CT, D>(a, k);
        struct Two {                             // entries of the two tiles of a step
            int a, b;
        };
        auto entries_at = [&](int kb) { return Two{entry_at(pl, kb), entry_at(pl, kb + 16)}; };
        auto load = [&](Tile<CT, D> (&raw)[2], const Two &e, int kb) {
            load_tile<CT, D, BUF_NT>(raw[0], chunks_at(pl, e.a, kb), kb & (P - 1), P, lane);
            load_tile<CT, D, BUF_NT>(raw[1], chunks_at(pl, e.b, kb + 16), (kb + 16) & (P - 1), P, lane);
        };
        Query<D> x[QT];
        bool whole_pages;
        auto compute = [&](Tile<CT, D> (&raw)[2], int kb) {
            f4 s[QT][2];
            auto scores = [&](const Tile<CT, D> &tile, int T) {
#pragma unroll
                for (int i = 0; i < QT; i++)
                    s[i][T] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int b = 0; b < G::NB; b++) {
                    if constexpr (FINE) {
                        const Frag c = key_codes<CT, D>(tile, b);
                        const h2 dd = key_scale<CT, D>(tile, b);
                        Frag hi, lo;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            hi.p[i] = c.p[i] * dd;
                            lo.p[i] = __builtin_elementwise_fma(c.p[i], dd, -hi.p[i]);
                        }
#pragma unroll
                        for (int i = 0; i < QT; i++) {
                            s[i][T] = mfma(hi.v, x[i].q[b], s[i][T]);
                            s[i][T] = mfma(lo.v, x[i].q[b], s[i][T]);
                        }
                    } else {
                        const h8 kf = key_frag<CT, D>(tile, b);
#pragma unroll
                        for (int i = 0; i < QT; i++)
                            s[i][T] = mfma(kf, x[i].q[b], s[i][T]);
                    }
                }
            };
            scores(raw[0], 0);
            scores(raw[1], 1);
            if (kb + STEP > pl.plain || !whole_pages) {
                // some keys are new tokens, past the end or on no page
                const bool oka = mapped(pl, entry_at(pl, kb), kb);
                const bool okb = mapped(pl, entry_at(pl, kb + 16), kb + 16);
#pragma unroll
                for (int i = 0; i < QT; i++)
                    mask_scores<D>(s[i], x[i], arguments().a, w, kb, oka, okb, g);
                drop_values<CT, D>(raw[0], kb + 4 * g, oka, w.ctx, w.L);
                drop_values<CT, D>(raw[1], kb + 16 + 4 * g, okb, w.ctx, w.L);
            }
            h8 pr[QT], rest[QT];
#pragma unroll
            for (int i = 0; i < QT; i++)
                pr[i] = softmax_step<D, FINE>(s[i], x[i], rest[i]);
#pragma unroll
            for (int t = 0; t < G::NT; t++) {
                Frag f;
                value_half<CT, D>(raw[0], t, f.p[0], f.p[1]);
                value_half<CT, D>(raw[1], t, f.p[2], f.p[3]);
#pragma unroll
                for (int i = 0; i < QT; i++) {
                    x[i].o[t] = mfma(f.v, pr[i], x[i].o[t]);
                    if constexpr (FINE)
                        x[i].o[t] = mfma(f.v, rest[i], x[i].o[t]);
                }
            }
        };

        // one step computed, the next one's codes on their way, and the page
        // numbers of the one after that
        int kb = k.begin + wave * STEP;
        Tile<CT, D> ra[2], rb[2];
        load(ra, entries_at(kb), kb);
        Two en = entries_at(kb + STRIDE);
        whole_pages = all_mapped(pl, k.begin, lane);
#pragma unroll
        for (int i = 0; i < QT; i++)
            load_query<D>(x[i], a, w, QT, i, lane);
        for (; kb < k.end; kb += 2 * STRIDE) {
            load(rb, en, kb + STRIDE);
            en = entries_at(kb + 2 * STRIDE);
            compute(ra, kb);
            load(ra, en, kb + 2 * STRIDE);
            en = entries_at(kb + 3 * STRIDE);
            compute(rb, kb + STRIDE);            // past the end no key is seen
        }
        finish<CT, D, QT, 1, WAVES>(x, arguments(), k, 0, wave, lane, red, ml);
    }
}

// More rows: W waves, RG groups of them with QT * 16 rows each, KG = W / RG
// waves per group.  16 W keys at a time lie dequantized in LDS, as the fragments
// of the matrix instructions; each wave reads its group's share of them (STEPS
// times 32 keys) and meanwhile dequantizes a 16-key tile of the next ones into
// a second buffer, between its matrix instructions, so that one barrier a step
// is enough; the codes after those are on their way.
template <int CT, int D, int QT, int RG, int W, bool FINE>
__global__ __launch_bounds__(64 * W, D <= 128 ? 2 : 1) void k_attn_rows(Launch launch)
{
    using G = Geo<CT, D>;
    constexpr int KEYS = 16 * W, KG = W / RG, STEPS = W / 2 / KG, AUX = RG == 2 ? BUF_NT : 0;
    constexpr int K_FRAGS = W * G::NB, V_FRAGS = W / 2 * G::NT;
    constexpr int STAGE = (K_FRAGS + V_FRAGS) * 64, JOIN = W * RED * 64;
    __shared__ h8 lds[2 * STAGE > JOIN ? 2 * STAGE : JOIN];
    __shared__ float ml[W * QT * 16 * 2];
    __shared__ __align__(16) float key_scales[FINE ? 2 * G::NB * KEYS : 4];
    const int lane0 = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int rg = wave / KG, kg = wave % KG;
    const int P = 1 << launch.a.log_page;
    Cursor cur = first_span(launch.a, launch.p, KEYS, lane0);
    Work k;
    for (bool first = true; next_work(cur, k, arguments(), KEYS, first); first = false) {
        const Rows &w = k.w;
        const AttnArgs &a = arguments().a;
        const int lane = fresh(lane0), g = lane >> 4;
        const Place pl = place_of<CT, D>(a, k);
        Tile<CT, D> raw;
        // the wave's tile of the keys from kb
        auto chunks = [&](int entry, int kb) { return chunks_at(pl, entry, kb + 16 * wave); };
        auto entry = [&](int kb) { return entry_at(pl, kb + 16 * wave); };
        bool whole_pages;
        auto keep_values = [&](int kb) {
            if (kb + KEYS > pl.plain || !whole_pages) {
                const int key = kb + 16 * wave;
                drop_values<CT, D>(raw, key + 4 * g, mapped(pl, entry_at(pl, key), key), w.ctx, w.L);
            }
        };
        auto stage_key = [&](int turn, int b) {
            h8 *to = lds + turn * STAGE + (wave * G::NB + b) * 64 + lane;
            if constexpr (FINE) {
                *to = key_codes<CT, D>(raw, b).v;
                if (g == (b & 3))
                    key_scales[(turn * G::NB + b) * KEYS + 16 * wave + (lane & 15)] =
                        (float)key_scale<CT, D>(raw, b)[0];
            } else {
                *to = key_frag<CT, D>(raw, b);
            }
        };
        auto stage_value = [&](h8 *buf, int t) {
            union {
                h2 h[2];
                u2 u;
            } v;
            value_half<CT, D>(raw, t, v.h[0], v.h[1]);
            ((u2 *)&buf[(K_FRAGS + (wave >> 1) * G::NT + t) * 64 + lane])[wave & 1] = v.u;
        };

        load_tile<CT, D, AUX>(raw, chunks(entry(k.begin), k.begin), (k.begin + 16 * wave) & (P - 1), P,
                         lane);
        int en = entry(k.begin + KEYS);
        whole_pages = all_mapped(pl, k.begin, lane);
        Query<D> x[QT];
#pragma unroll
        for (int i = 0; i < QT; i++)
            load_query<D>(x[i], a, w, RG * QT, rg * QT + i, lane);
        keep_values(k.begin);
        __syncthreads();                         // the last rows' fragments are used up
#pragma unroll
        for (int b = 0; b < G::NB; b++)
            stage_key(0, b);
#pragma unroll
        for (int t = 0; t < G::NT; t++)
            stage_value(lds, t);
        load_tile<CT, D, AUX>(raw, chunks(en, k.begin + KEYS),
                         (k.begin + KEYS + 16 * wave) & (P - 1), P, lane);
        en = entry(k.begin + 2 * KEYS);
        int turn = 0;
        for (int kb = k.begin; kb < k.end; kb += KEYS, turn ^= 1) {
            const h8 *kf = lds + turn * STAGE, *vf = kf + K_FRAGS * 64;
            h8 *put = lds + (turn ^ 1) * STAGE;
            const Chunks ch = chunks(en, kb + 2 * KEYS);
            const int pos = (kb + 2 * KEYS + 16 * wave) & (P - 1);
            en = entry(kb + 3 * KEYS);
            keep_values(kb + KEYS);
            __syncthreads();
#pragma unroll
            for (int i0 = 0; i0 < STEPS; i0++) {
                const int n = kg * STEPS + i0, kp = kb + STEP * n;
                if (kp >= k.end)
                    continue;                    // then nothing is to be staged either
                const bool stage = i0 == 0;
                // all of a step's keys are asked for before the first product,
                // all of its values before the softmax: the reads' latency
                // passes behind them.  The products go before the other wave's
                // vector work on the same SIMD (4 sequences of 40000 Q4_0 keys,
                // 32 tokens: 107.6 us, 116 without)
                f4 s[QT][2];
                h8 kv[2 * G::NB], vv[G::NT];
#pragma unroll
                for (int b = 0; b < 2 * G::NB; b++)
                    kv[b] = kf[(2 * n * G::NB + b) * 64 + lane];
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int T = 0; T < 2; T++) {
#pragma unroll
                    for (int i = 0; i < QT; i++)
                        s[i][T] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int b = 0; b < G::NB; b++) {
                        if constexpr (FINE) {
                            const f4 d = *(const f4 *)&key_scales[(turn * G::NB + b) * KEYS +
                                                                  STEP * n + 16 * T + 4 * g];
#pragma unroll
                            for (int i = 0; i < QT; i++) {
                                const f4 part = mfma(kv[T * G::NB + b], x[i].q[b], f4{0, 0, 0, 0});
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    s[i][T][e] = fmaf(part[e], d[e], s[i][T][e]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < QT; i++)
                                s[i][T] = mfma(kv[T * G::NB + b], x[i].q[b], s[i][T]);
                        }
                        if (stage && T == b % 2)
                            stage_key(turn ^ 1, b);
                    }
                }
                __builtin_amdgcn_s_setprio(0);
                if (stage)
                    load_keys<CT, D, AUX>(raw, ch, pos, P, lane);
#pragma unroll
                for (int t = 0; t < G::NT; t++)
                    vv[t] = vf[(n * G::NT + t) * 64 + lane];
                __builtin_amdgcn_sched_barrier(0);
                if (kp + STEP > pl.plain || !whole_pages) {
                    const bool oka = mapped(pl, entry_at(pl, kp), kp);
                    const bool okb = mapped(pl, entry_at(pl, kp + 16), kp + 16);
#pragma unroll
                    for (int i = 0; i < QT; i++)
                        mask_scores<D>(s[i], x[i], arguments().a, w, kp, oka, okb, g);
                }
                h8 pr[QT], rest[QT];
#pragma unroll
                for (int i = 0; i < QT; i++)
                    pr[i] = softmax_step<D, FINE>(s[i], x[i], rest[i]);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int t = 0; t < G::NT; t++) {
#pragma unroll
                    for (int i = 0; i < QT; i++) {
                        x[i].o[t] = mfma(vv[t], pr[i], x[i].o[t]);
                        if constexpr (FINE)
                            x[i].o[t] = mfma(vv[t], rest[i], x[i].o[t]);
                    }
                    if (stage)
                        stage_value(put, t);
                }
                __builtin_amdgcn_s_setprio(0);
                if (stage)
                    load_values<CT, D, AUX>(raw, ch, pos, P, lane);
            }
        }
        finish<CT, D, QT, RG, KG>(x, arguments(), k, rg, kg, lane, (f4 *)lds, ml);
    }
}

// Joins the parts of a head and row block, rescaled to the largest reference
// so far.  A wave adds one fragment's parts in order, AHEAD of them and of their
// references and sums loaded together; with many parts (SHARED) the four waves
// of a workgroup take every fourth part of one fragment, and their sums are
// joined through LDS.  16 parts of one token: 3.9 us; with the references read
// before the parts 5.0.
template <int CT, int D, bool SHARED>
__global__ __launch_bounds__(THREADS) void k_attn_combine(AttnArgs a, AttnPlan p, Parts parts)
{
    constexpr int NT = D / 16, AHEAD = 4, BY = SHARED ? WAVES : 1;
    __shared__ f4 red[WAVES][64];
    __shared__ float2 redm[WAVES][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t per = (uint32_t)a.kv_heads * p.row_blocks, b = blockIdx.x / per;
    const uint32_t q = blockIdx.x - b * per;
    const int32_t *list = (const int32_t *)(parts.list + blockIdx.x);
    const int slot0 = load_uniform(list), n_parts = load_uniform(list + 1);
    Rows w = rows_of(a, (int)b);
    w.h = (int)(q / p.row_blocks);
    w.rb = (int)(q - w.h * p.row_blocks);
    const int F = p.tiles * NT, ff = SHARED ? blockIdx.y : blockIdx.y * WAVES + wave;
    // rows that do not exist have no entry in the list
    if (w.rb >= blocks_of(a, p, w) || n_parts <= 1 || ff >= F)
        return;
    const int tile = ff / NT, ms = p.tiles * 16;
    const float2 *mlp = parts.ml + tile * 16 + (lane & 15);
    const f4 *o = parts.sum + ff * 64 + lane;
    auto slot = [&](int n) { return (int64_t)(n ? (slot0 | 1) - 1 + 2 * n : slot0); };
    float mm = NO_REF, ll = 0.0f;
    f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if ((w.rb * p.tiles + tile) * 16 + (lane & 15) < w.T * a.group) {
        for (int n0 = SHARED ? wave : 0; n0 < n_parts; n0 += AHEAD * BY) {
            float2 t[AHEAD];
            f4 v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; i++) {
                const int64_t at = slot(min(n0 + i * BY, n_parts - 1));
                t[i] = mlp[at * ms];
                v[i] = o[at * F * 64];
            }
            float top = mm;
#pragma unroll
            for (int i = 0; i < AHEAD; i++)
                top = n0 + i * BY < n_parts ? fmaxf(top, t[i].x) : top;
            const float f = __builtin_amdgcn_exp2f(mm - top);
            mm = top;
            ll *= f;
            sum *= f;
#pragma unroll
            for (int i = 0; i < AHEAD; i++)
                if (n0 + i * BY < n_parts) {
                    const float fi = __builtin_amdgcn_exp2f(t[i].x - top);
                    ll += fi * t[i].y;
                    sum += fi * v[i];
                }
        }
    }
    if constexpr (SHARED) {
        red[wave][lane] = sum;
        redm[wave][lane] = make_float2(mm, ll);
        __syncthreads();
        if (wave)
            return;
        for (int i = 0; i < WAVES; i++)
            mm = fmaxf(mm, redm[i][lane].x);
        ll = 0.0f;
        sum = f4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < WAVES; i++) {
            const float f = __builtin_amdgcn_exp2f(redm[i][lane].x - mm);
            ll += f * redm[i][lane].y;
            sum += f * red[i][lane];
        }
    }
    store_frag<CT, D>(a, w, p.tiles, tile, ff % NT, lane,
                      ll == 0.0f ? f4{0, 0, 0, 0} : sum * (1.0f / ll));
}

// Row tiles per wave with more than 32 rows: two share each fragment read;
// with 256 elements a head the registers hold one.
constexpr int rows_qt(int D) { return D <= 128 ? 2 : 1; }

template <int CT, int D, bool FINE>
void launch_steps(const Launch &args, dim3 grid, hipStream_t s)
{
    constexpr int QT = rows_qt(D);
    const AttnPlan &p = args.p;
    if (p.row_groups > 1 && p.waves == 4) {
        if (p.row_groups == 4)
            k_attn_rows<CT, D, QT, 4, 4, FINE><<<grid, 256, 0, s>>>(args);
        else
            k_attn_rows<CT, D, QT, 2, 4, FINE><<<grid, 256, 0, s>>>(args);
    } else if (p.row_groups > 1) {
        if constexpr (D <= 128) {
            if (p.row_groups == 4)
                k_attn_rows<CT, D, QT, 4, 8, FINE><<<grid, 512, 0, s>>>(args);
            else
                k_attn_rows<CT, D, QT, 2, 8, FINE><<<grid, 512, 0, s>>>(args);
        }
    } else if (p.tiles == 1) {
        k_attn<CT, D, 1, FINE><<<grid, THREADS, 0, s>>>(args);
    } else if constexpr (D <= 128) {
        k_attn<CT, D, 2, FINE><<<grid, THREADS, 0, s>>>(args);
    }
}

// Workgroups of an uncut launch: all sequences with the row blocks that
// max_nodes asks for, or (by_rows) no more row blocks than `tokens` rows can
// fill, one begun for each sequence.  Below 2^27 within the limits of the entry
// point; the second grid dimension holds what the first does not.
int64_t unit_count(const AttnArgs &a, const AttnPlan &p)
{
    return a.kv_heads * (p.by_rows ? a.tokens * a.group / (p.tiles * 16) + a.batch
                                   : (int64_t)a.batch * p.row_blocks);
}

dim3 unit_grid(int64_t units)
{
    constexpr int64_t X = 1 << 20;
    return units <= X ? dim3((unsigned)units) : dim3((unsigned)X, (unsigned)((units + X - 1) / X));
}

template <int CT, int D>
hipError_t launch_cd(const AttnArgs &a, const AttnPlan &p, void *scratch, hipStream_t s)
{
    const int64_t units = (int64_t)a.batch * a.kv_heads * p.row_blocks;
    const dim3 grid = p.groups ? dim3((unsigned)p.groups) : unit_grid(unit_count(a, p));
    if (!grid_fits(grid.x, 64 * p.waves))
        return hipErrorInvalidConfiguration;
    const int F = p.tiles * (D / 16);
    Parts parts{nullptr, nullptr, nullptr};
    if (p.groups > 1) {
        parts.sum = (f4 *)scratch;
        parts.ml = (float2 *)(parts.sum + (size_t)2 * p.groups * F * 64);
        parts.list = (int2 *)(parts.ml + (size_t)2 * p.groups * p.tiles * 16);
    }
    const Launch args{a, p, parts};
    if (a.dtype == TQ_F16)
        launch_steps<CT, D, true>(args, grid, s);
    else
        launch_steps<CT, D, false>(args, grid, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.groups <= 1)
        return e;
    if (p.groups >= 16 * units)
        k_attn_combine<CT, D, true><<<dim3((unsigned)units, (unsigned)F), THREADS, 0, s>>>(a, p, parts);
    else
        k_attn_combine<CT, D, false><<<dim3((unsigned)units, (unsigned)((F + WAVES - 1) / WAVES)),
                                       THREADS, 0, s>>>(a, p, parts);
    return hipGetLastError();
}

template <int CT>
hipError_t launch_c(int D, const AttnArgs &a, const AttnPlan &p, void *scratch, hipStream_t s)
{
    switch (D) {
    case 64: return launch_cd<CT, 64>(a, p, scratch, s);
    case 96: return launch_cd<CT, 96>(a, p, scratch, s);
    case 128: return launch_cd<CT, 128>(a, p, scratch, s);
    case 256: return launch_cd<CT, 256>(a, p, scratch, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

AttnPlan attn_plan(int D, int64_t batch, int64_t heads, int64_t kv_heads, int64_t max_nodes,
                   int64_t max_keys, bool even)
{
    AttnPlan p{};
    const int64_t rows = max_nodes * (heads / kv_heads);
    const int qt = rows_qt(D);
    if (rows <= 16) {
        p.row_groups = 1;
        p.tiles = 1;
    } else if (rows <= 32 && D <= 128) {
        p.row_groups = 1;
        p.tiles = 2;
    } else {
        p.row_groups = rows <= 32 * qt ? 2 : 4;
        p.tiles = p.row_groups * qt;
    }
    p.row_blocks = (int)((rows + 16 * p.tiles - 1) / (16 * p.tiles));
    const int64_t units = batch * kv_heads * p.row_blocks;
    // Two workgroups of four waves for each of 256 compute units, or one of
    // eight; one of four where a head is wider than 128 (256 elements, 4
    // sequences of 8192 keys, 32 tokens: 65.9 us, with two a unit in the line
    // 80.5).  That is what fits with 16 and more rows of heads of 96 and 128; by
    // their registers, one row tile of 64 elements would leave room for four a
    // unit, of 96 and 128 in Q4_0 for three, of 256 in Q4_0 for two.  One token
    // for each of 64 sequences of 8192 keys reads 6.0 (64, Q8_0), 4.0 (64, Q4_0),
    // 5.7 (128, Q4_0) and 5.7 TB/s (256, Q4_0) so, 6.4 with 128 in Q8_0.
    p.waves = p.row_groups > 1 && D <= 128 && units <= FEW_UNITS ? 8 : 4;
    const int keys = p.waves * (p.row_groups > 1 ? 16 : STEP), least = MIN_KEYS / keys;
    const int64_t line = units * ((max_keys + keys - 1) / keys + least);
    p.groups = units >= (even ? EVEN_UNITS : OWN_UNITS)
                   ? 0
                   : (int)std::min<int64_t>(D > 128 || p.waves == 8 ? 256 : 512,
                                            std::max<int64_t>(1, line / least));
    return p;
}

size_t attn_scratch_bytes(const AttnPlan &p, int D, int64_t batch, int64_t kv_heads)
{
    if (p.groups <= 1)
        return 0;
    return (size_t)2 * p.groups * p.tiles * ((size_t)(D / 16) * 1024 + 16 * sizeof(float2)) +
           (size_t)batch * kv_heads * p.row_blocks * sizeof(int2);
}

hipError_t launch_attention(int cache_type, int D, const AttnArgs &a, const AttnPlan &plan,
                            void *scratch, hipStream_t s)
{
    AttnPlan p = plan;
    p.by_rows = 1;
    const int64_t by_rows = unit_count(a, p);
    p.by_rows = 0;
    p.by_rows = p.groups == 0 && by_rows < unit_count(a, p);
    return cache_type == TQ_Q8_0 ? launch_c<TQ_Q8_0>(D, a, p, scratch, s)
                                 : launch_c<TQ_Q4_0>(D, a, p, scratch, s);
}

}  // namespace tq
