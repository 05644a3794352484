// Host-side hooks of the training operators' translation units.
#pragma once

namespace psk {

// The resident loss kernel's status word (read, then zeroed if `reset`) and its
// copy of the lost-copy test hook.
int loss_status(unsigned int* v, bool reset);
int loss_set_drop_row(long long row);

}  // namespace psk
