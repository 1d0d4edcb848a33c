// How the boundary's backward deals its rows out to teams (plain C++).
#pragma once

#include <stdint.h>

namespace mtgr {

// Gradient slots of the workspace, per team and group.
constexpr int kSlots = 5;

// Rows of a team, the last one's fewer: in 64 bits, T may be any int32.
inline int32_t rows_per_team(int32_t T, int32_t teams) { return (int32_t)(((int64_t)T + teams - 1) / teams); }

// Teams of the backward: at most `resident`, at least 4 rows each, and at most
// 256 MB of gradient slots.
inline int32_t bwd_teams(int32_t T, int32_t d, int32_t G, int64_t resident) {
  if (T <= 0) return 0;
  int64_t teams = resident;
  const int64_t most = (256ll << 20) / ((int64_t)G * kSlots * d * 4);
  if (teams > most) teams = most > 0 ? most : 1;
  const int64_t by_rows = ((int64_t)T + 3) / 4;
  if (teams > by_rows) teams = by_rows;
  const int64_t rows = ((int64_t)T + teams - 1) / teams;
  return (int32_t)(((int64_t)T + rows - 1) / rows);
}

}  // namespace mtgr
