// What the kernels of a step with shared prefixes hand to one another: the plan
// writes it, in the caller's workspace.
#pragma once

#include "kernels.h"

namespace cb {

// A row's state over a part of its keys is a record: acc[kPrefixDim], the sum of
// 2^(s - m) v over scores s in the exp2 domain, and apart from it (so that acc
// fills whole lines) the reference maximum m and the sum of 2^(s - m).
constexpr int kPrefixDim = 128;
constexpr int kPrefixRecBytes = (kPrefixDim + 2) * 4;

// A piece: the query rows of one row tile or two, of one key/value head, over one
// KV segment, either of their group's prefix or of their sequence's own keys.
struct alignas(16) Piece {
  int s0;                      // the table that names the blocks (a group's first sequence's, or the own one)
  int skip;                    // blocks of it before key 0
  int tok0, ntok;              // query tokens
  int hk;                      // key/value head
  int j0, nt;                  // KV tiles (none: the rows' records are empty)
  int keys;                    // keys of the prefix, or own keys of the sequence
  int lim0;                    // keys that the first token sees; the next one sees one more, up to `keys`
  unsigned rec0;               // record of (tok0, head 0)
  int rec_step;                // records per (token, head)
  int flags;
  int pad[4];
};
static_assert(sizeof(Piece) == 64, "piece");
enum : int {
  kPieceAlt = 1,               // one row tile: KV tiles alternate over the two slots, which have a record each
  kPieceDirect = 2,            // nothing to join: the rows are written to out
  kPieceEnd = 4                // no more pieces
};

// One row tile of a sequence over one chunk of its own keys, for every key/value head.
struct alignas(16) SuffixItem {
  int s;
  int tok0, q_len;             // the sequence's packed rows
  int row0;                    // first row of the tile (row = token * G + head of the group)
  int k0, k1;                  // own keys of the chunk (0 = the first key behind the prefix)
  int ctx;                     // own keys of the sequence
  int skip;                    // blocks of the table that the prefix covers
  unsigned rec0;               // the chunk's record of (the sequence's first token, head 0)
  int rec_step;                // records per (token, head)
  int direct;                  // 1: nothing to join, the rows are written to out
  int pad;                     // the plan's counter
};
static_assert(sizeof(SuffixItem) == 48, "item");

struct PrefixWork {
  const int32_t* cu_groups;    // [num_groups + 1]
  const int32_t* prefix_lens;  // [num_groups]
  const int32_t* context_lens; // [num_seqs], whole
  int32_t num_groups;
  int32_t num_sms;
  int32_t tile_tokens;         // query tokens per row tile of a piece
  int32_t stream_units;        // streamed units that the chunk length aims for
  int32_t min_chunk_tiles;     // shortest chunk of a small step's streams, in 16-key tiles
  int32_t max_sharers;         // sequences that could share, up to which the small step's kernel runs the step and
                               // beyond which it leaves it to the plan's behind it; -1: one of them is launched
  int32_t piece_cap, item_cap;
  int64_t prefix_rec_cap;      // records of the prefixes; the own ones follow
  int64_t piece_rec_cap;       // own records of pieces
  int64_t own_rec_cap;         // all own records
  uint32_t tag;
  // in the workspace
  int32_t* header;             // [0] pieces, [1] prefix records per row (stride), [2] call tag, [3] piece
                               // claims, [4] streamed items, [5] unit claims, [6] CTAs that work on
                               // pieces first (the others go to the streamed units at once), [7] where both
                               // are launched: 1 if the small step's kernel runs the step, else 0
  int4* groups;                // [num_groups], [num_seqs], [num_groups + num_seqs]: the plan's own, where
  int4* seqs;                  // they do not fit its shared memory
  int32_t* first_piece;
  int4* seq_recs;              // [num_seqs] as token_info, of the sequence's first token
  Piece* pieces;
  SuffixItem* items;
  int4* token_info;            // [num_tokens] (prefix records, first own record of head 0, own records per head, -)
  float* recs;                 // acc of the prefix records [token][query head][stride], then the sequences' own ones
  float2* rec_ml;              // (m, sum) of the same
};

constexpr int kStreamWarps = 8;          // warps of a CTA that stream own keys, each with units of its own

}  // namespace cb
