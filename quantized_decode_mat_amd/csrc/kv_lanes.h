// kv_lanes.h — which elements of a token's row each lane of the single-token
// attention kernel loads, and which threads add up its join. Plain constant
// expressions: the kernel and a check on the host, lane by lane, use the same
// ones.
#pragma once

namespace xq {

// Dims are padded to the next of these; the operands' lanes are laid out for
// the padded row.
constexpr int decode_dim_pad(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

// K: four groups of 16 lanes take 16 bytes each of a row, `decode_k_loads`
// times. The first element of group lg's load s, by its place in the padded
// row; past a shorter row's end it is the row's first.
constexpr int decode_k_loads(int dp, int elem_bytes) { return dp * elem_bytes / 64; }
template <int DP, bool FULL>
constexpr int decode_k_dim(int s, int lg, int elem_bytes, int dim) {
  const int d0 = (s * 4 + lg) * (16 / elem_bytes);
  return FULL || d0 < dim ? d0 : 0;
}

// V: 16 lanes take decode_v_dims elements each, decode_v_loads times. The last
// round of 192 dims has lanes past even a full row's end (16 x 8 x 2 is 256):
// only where the rounds fill the row is no comparison needed.
constexpr int decode_v_dims(int dp) { return dp == 64 ? 4 : 8; }
constexpr int decode_v_loads(int dp) { return (dp + 16 * decode_v_dims(dp) - 1) / (16 * decode_v_dims(dp)); }
template <int DP, bool FULL>
constexpr int decode_v_dim(int c, int l16, int dim) {
  constexpr bool kFits = FULL && decode_v_loads(DP) * 16 * decode_v_dims(DP) == DP;
  const int d0 = (c * 16 + l16) * decode_v_dims(DP);
  return kFits || d0 < dim ? d0 : 0;
}

// The join's `quads` outputs of four, more than threads or fewer: a round's
// thread t adds to output t / teams, every teams-th part, and the first thread
// of each team then adds the team's sums (those of the `teams` threads from t
// on). Threads past teams * quads have no output.
constexpr int join_teams(int threads, int quads) { return threads > quads ? threads / quads : 1; }
constexpr bool join_adds(int t, int teams, int quads) { return t % teams == 0 && t / teams < quads; }

}  // namespace xq
