// Layout of the paged block-quantized key / value cache (tq_cache_write,
// tq_cache_read, tq_tree_attention).
//
// A cache buffer is [page][kv head] chunks of page_size tokens; a chunk is
// all its codes, then all its fp16 scales.  Codes are unsigned: Q8_0 code +
// 128 in a byte, Q4_0 the nibble 0..15 (code + 8).  The orders inside a
// chunk are those in which one lane of the attention's 16x16x32 fp16 matrix
// instructions wants its operand, so that codes go from memory to the matrix
// cores through registers alone:
//
//   K codes  [token / 16][piece][lane group][token % 16]: lane group g (0..3)
//            of an instruction holds elements 8g..8g+7 of a 32-element block.
//            Eight elements are 8 bytes (Q8_0) or 4 (Q4_0); a piece is those of
//            consecutive blocks, up to 16 bytes (k_piece).  A wave that loads
//            a piece of 16 tokens reads consecutive bytes in lane order.
//   K scales [token][D / 32].
//   V codes  [token / 4][column][token % 4]: 4 tokens of one element (Q8_0:
//            column = element) or of an element pair (Q4_0: column c holds
//            elements 2c, 2c + 1 in the low / high nibble) in a dword, because
//            the product with the probabilities contracts over tokens.
//   V scales [D / 32][token].
//
// Nibbles and bytes are placed so that the pairs that (w >> 4j) & 0x000f000f
// picks out are neighbours in the operand: element i of a Q4_0 K piece is
// nibble k4_shift(i), token t of a Q4_0 V dword is byte v4_byte(t).
#pragma once

#include <stdint.h>

#include "tiledq.h"

namespace tq {

constexpr bool cache_type_ok(int ct) { return ct == TQ_Q8_0 || ct == TQ_Q4_0; }
constexpr bool cache_dim_ok(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 256; }
constexpr bool cache_page_ok(int64_t P) { return P >= 16 && P <= 1024 && (P & (P - 1)) == 0; }

// Bytes of the codes of one token of one head, and of one [page][head] chunk.
constexpr int64_t token_code_bytes(int ct, int64_t D) { return ct == TQ_Q8_0 ? D : D / 2; }
constexpr int64_t chunk_bytes(int ct, int64_t D, int64_t P)
{
    return P * (token_code_bytes(ct, D) + D / 16);
}

// Bytes of a piece of K codes: 16 where D gives whole ones, else all of a
// lane group's blocks (Q4_0) or one (Q8_0).
template <int CT, int D> constexpr int k_piece()
{
    if (CT == TQ_Q8_0)
        return D % 64 == 0 ? 16 : 8;
    return D % 128 == 0 ? 16 : D / 8;
}

// Byte offset, within a chunk, of the codes of lane group g of block s of the
// token at position pos.
template <int CT, int D> __host__ __device__ constexpr int k_offset(int pos, int s, int g)
{
    constexpr int TB = (int)token_code_bytes(CT, D), B = k_piece<CT, D>();
    constexpr int one = CT == TQ_Q8_0 ? 8 : 4, per = B / one;
    return (pos >> 4) * (16 * TB) + (s / per) * (64 * B) + (g * 16 + (pos & 15)) * B + s % per * one;
}

// Bit position of element i (0..7) in a Q4_0 K piece.
__host__ __device__ constexpr int k4_shift(int i)
{
    const int f = i >> 1, h = i & 1;
    return 8 * (2 * h + (f >> 1)) + 4 * (f & 1);
}

// Byte of token t (0..3) in a Q4_0 V dword.
__host__ __device__ constexpr int v4_byte(int t) { return ((t & 1) << 1) | (t >> 1); }

}  // namespace tq
