// kd_rope.h -- shared by the rotating entry points (library internal).
#pragma once
#include "kd.h"

namespace kd {
// KD_OK where t is a table as kd_rope_plan makes it.
kd_status rope_table_check(const char* fn, const kd_rope_table* t);
}  // namespace kd
